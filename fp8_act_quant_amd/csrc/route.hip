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

typedef float f32x4 __attribute__((ext_vector_type(4)));

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

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t umin(uint32_t a, uint32_t b) { return a < b ? a : b; }

// Order-preserving integer key of a number: a > b as floats is key(a) > key(b) as unsigned. Every key
// is above 0 (that of the NaN of all ones by the maximum); 0 stands for "no candidate", so that top_k
// candidates are found whatever the logits hold. (A choice is never -0: scores are +0 at the least,
// and +0 + -0 = +0.)
__device__ __forceinline__ uint32_t key_of(float c) {
    const uint32_t u = __float_as_uint(c);
    return umax(u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u), 1u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// v of another lane of the same 16 (all of whose lanes are active)
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kMirror8 = 0x141, kMirror16 = 0x140;

// maximum over 16 lanes, in each of them
__device__ __forceinline__ uint32_t team_max(uint32_t v) {
    v = umax(v, dpp<kXor1>(v));
    v = umax(v, dpp<kXor2>(v));
    v = umax(v, dpp<kMirror8>(v));
    return umax(v, dpp<kMirror16>(v));
}
// and over the wave's 64
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = team_max(v);
    v = umax(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, false));   // row_bcast15
    v = umax(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, false));   // row_bcast31
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

__device__ __forceinline__ float read_f(float v, int lane) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}
template <int CTRL>
__device__ __forceinline__ float dpp_f(float v) { return __uint_as_float(dpp<CTRL>(__float_as_uint(v))); }
__device__ __forceinline__ float team_max(float v) {
    v = fmaxf(v, dpp_f<kXor1>(v));
    v = fmaxf(v, dpp_f<kXor2>(v));
    v = fmaxf(v, dpp_f<kMirror8>(v));
    return fmaxf(v, dpp_f<kMirror16>(v));
}
__device__ __forceinline__ float wave_max(float v) {
    v = team_max(v);
    return fmaxf(fmaxf(read_f(v, 0), read_f(v, 16)), fmaxf(read_f(v, 32), read_f(v, 48)));
}

// sums over 16 lanes or the wave's 64, in a fixed order and the same in every lane
__device__ __forceinline__ float team_sum(float v) {
    v += dpp_f<kXor1>(v);
    v += dpp_f<kXor2>(v);
    v += dpp_f<kMirror8>(v);
    return v + dpp_f<kMirror16>(v);
}
__device__ __forceinline__ float wave_sum(float v) {
    v = team_sum(v);
    return (read_f(v, 0) + read_f(v, 16)) + (read_f(v, 32) + read_f(v, 48));
}
template <int CTRL>
__device__ __forceinline__ double dpp_d(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, (uint64_t)dpp<CTRL>((uint32_t)u) | (uint64_t)dpp<CTRL>((uint32_t)(u >> 32)) << 32);
}
__device__ __forceinline__ double read_d(double v, int lane) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
    return __builtin_bit_cast(double, (uint64_t)lo | (uint64_t)hi << 32);
}
__device__ __forceinline__ double team_sum(double v) {
    v += dpp_d<kXor1>(v);
    v += dpp_d<kXor2>(v);
    v += dpp_d<kMirror8>(v);
    return v + dpp_d<kMirror16>(v);
}
__device__ __forceinline__ double wave_sum(double v) {
    v = team_sum(v);
    return (read_d(v, 0) + read_d(v, 16)) + (read_d(v, 32) + read_d(v, 48));
}

template <int BF16>
__device__ __forceinline__ float load_logit(const void *p, int64_t i) {
    if constexpr (BF16) return __uint_as_float((uint32_t) reinterpret_cast<const uint16_t *>(p)[i] << 16);
    else return reinterpret_cast<const float *>(p)[i];
}

// V consecutive elements from row + first, n of which belong to this lane (what the others hold is
// some element of the row). FULL: n is V or at most 0 and rows are aligned to V elements, so they
// come in one load. Every lane loads, without a branch.
template <int V, int BF16, int FULL>
__device__ __forceinline__ void load_row(const void *p, int64_t row, int first, int n, int E, float (&x)[V]) {
    if constexpr (FULL) {
        const int i = n > 0 ? first : 0;
        if constexpr (BF16) {
            typedef uint16_t piece __attribute__((ext_vector_type(V)));
            const piece u = *reinterpret_cast<const piece *>(reinterpret_cast<const uint16_t *>(p) + row + i);
#pragma unroll
            for (int j = 0; j < V; ++j) x[j] = __uint_as_float((uint32_t)u[j] << 16);
        } else {
            typedef float piece __attribute__((ext_vector_type(V)));
            const piece u = *reinterpret_cast<const piece *>(reinterpret_cast<const float *>(p) + row + i);
#pragma unroll
            for (int j = 0; j < V; ++j) x[j] = u[j];
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) x[j] = load_logit<BF16>(p, row + min(first + j, E - 1));
    }
}
// The same where a lane's elements are whole quads of an aligned row
template <int V, int BF16>
__device__ __forceinline__ void load_quads(const void *p, int64_t row, int first, int n, float (&x)[V]) {
#pragma unroll
    for (int j = 0; j < V; j += 4) {
        float quad[4];
        load_row<4, BF16, 1>(p, row, first + j, n - j, 0, quad);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[j + i] = quad[i];
    }
}
// whether element j of a lane's V is one of its n
template <int FULL>
__device__ __forceinline__ bool has(int j, int n) {
    return FULL ? n > 0 : j < n;
}

// 1 / (1 + exp(-x)) with every step rounded to nearest. The quotient is v_rcp_f32 and one
// Newton step, which gives the correctly rounded reciprocal of a float in [1, 2^126) (the tests
// hold 12 million logits' scores to the division, bit for bit), in 3 operations instead of a
// division's 10; past that (x < -87) the division itself is taken.
template <int V>
__device__ __forceinline__ void sigmoid(const float (&x)[V], float (&s)[V]) {
    float d[V], most = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        d[i] = 1.0f + expf(-x[i]);
        const float y = __builtin_amdgcn_rcpf(d[i]);
        s[i] = __builtin_fmaf(__builtin_fmaf(-d[i], y, 1.0f), y, y);
        most = fmaxf(most, d[i]);   // (a NaN is left out here, and comes out as one either way)
    }
    if (__any(most >= 0x1p126f)) {
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] = d[i] < 0x1p126f ? s[i] : 1.0f / d[i];
    }
}

// softmax's maximum and denominator from each lane's values (-inf where there is none);
// total = 0 when no value is above -inf, and every score is then 0. e: the numerators.
template <int V, int TEAM>
__device__ __forceinline__ void softmax_of(const float (&x)[V], float (&e)[V], float &top, float &total) {
    float m = x[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = fmaxf(m, x[i]);
    top = TEAM ? team_max(m) : wave_max(m);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        e[i] = expf(x[i] - top);
        sum += (double)e[i];
    }
    total = top == -__builtin_inff() ? 0.0f : (float)(TEAM ? team_sum(sum) : wave_sum(sum));
}

// The scores of a lane's logits; top and total are softmax's. e / total is rounded to nearest:
// Markstein's two corrections on the rounded reciprocal, which are exact while their residual
// does not underflow (e >= 2^-90, or 0); smaller ones take the division.
template <int V, int SOFTMAX, int TEAM = 0>
__device__ __forceinline__ void scores(const float (&x)[V], float (&s)[V], float &top, float &total) {
    if constexpr (SOFTMAX) {
        float e[V];
        softmax_of<V, TEAM>(x, e, top, total);
        const float y = 1.0f / total;
        bool far = false;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float q = e[i] * y;
            s[i] = __builtin_fmaf(__builtin_fmaf(-q, total, e[i]), y, q);
            far |= e[i] != 0.0f && !(e[i] >= 0x1p-90f);
        }
        if (__any(far) || !(total > 0.0f)) {
#pragma unroll
            for (int i = 0; i < V; ++i) s[i] = total > 0.0f ? e[i] / total : 0.0f;
        }
    } else {
        sigmoid<V>(x, s);
    }
}

// One logit's score, given them
template <int SOFTMAX>
__device__ __forceinline__ float score_of(float x, float top, float total) {
    if constexpr (SOFTMAX) {
        return total > 0.0f ? expf(x - top) / total : 0.0f;
    } else {
        const float in[1] = {x};
        float out[1];
        sigmoid<1>(in, out);
        return out[0];
    }
}

// The two largest keys of the group's lanes, from each lane's two
__device__ __forceinline__ void merge2(uint32_t &m1, uint32_t &m2, uint32_t o1, uint32_t o2) {
    m2 = umax(umax(m2, o2), umin(m1, o1));
    m1 = umax(m1, o1);
}

// One wave per token. Lane l belongs to group l >> lane_shift and holds V consecutive experts
// of it, so lane order is expert order, and a reduction over a group is one over a power of
// two of adjacent lanes. Each lane sorts its keys (V <= 8; equal ones keep their order), so a
// selected expert is always some lane's first: a maximum over the first ones, then that lane
// moves up. About 20 operations per selected expert; with more experts a lane the sorting
// would cost more than it saves, and each step looks at all of them. Bound by these operations
// (some 400 a token), not by the 4 E bytes it reads: 16384 tokens' 256 experts 13.0 us, 1.4 TB/s.
template <int V, int BF16, int SOFTMAX, int FULL>
__global__ __launch_bounds__(64 * kWaves) void route_kernel(RouteArgs a) {
    typedef float piece __attribute__((ext_vector_type(V)));
    __shared__ piece rows[kWaves][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t = (int64_t)blockIdx.x * kWaves + wave;
    if (t >= a.T) return;
    const int lanes = 1 << a.lane_shift;
    const int group = lane >> a.lane_shift;
    const int at = (lane & (lanes - 1)) * V;                          // first expert within the group
    const int n = group < a.groups ? max(min(a.per - at, V), 0) : 0;  // experts of this lane
    const int e0 = group * a.per + at;
    const int64_t row = t * a.E;

    float x[V], s[V], bias[V], top = 0.0f, total = 1.0f;
    load_row<V, BF16, FULL>(a.logits, row, e0, n, a.E, x);
#pragma unroll
    for (int i = 0; i < V; ++i) bias[i] = 0.0f;
    if (a.bias) load_row<V, 0, FULL>(a.bias, 0, e0, n, a.E, bias);
    if constexpr (SOFTMAX) {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = has<FULL>(i, n) ? x[i] : -__builtin_inff();
    }
    scores<V, SOFTMAX>(x, s, top, total);
    uint32_t key[V];
    piece kept_scores;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const uint32_t k = key_of(s[i] + bias[i]);
        key[i] = has<FULL>(i, n) ? k : 0u;
        kept_scores[i] = s[i];
    }
    rows[wave][lane] = kept_scores;   // lane l's i-th expert is place l * V + i

    if (a.groups > 1) {
        uint32_t m1 = key[0], m2 = 0;   // the two largest keys of the group
#pragma unroll
        for (int i = 1; i < V; ++i) merge2(m1, m2, key[i], 0);
        if (lanes > 1) merge2(m1, m2, dpp<kXor1>(m1), dpp<kXor1>(m2));
        if (lanes > 2) merge2(m1, m2, dpp<kXor2>(m1), dpp<kXor2>(m2));
        if (lanes > 4) merge2(m1, m2, dpp<kMirror8>(m1), dpp<kMirror8>(m2));
        if (lanes > 8) merge2(m1, m2, dpp<kMirror16>(m1), dpp<kMirror16>(m2));
        if (lanes > 16) merge2(m1, m2, __shfl_xor(m1, 16, 64), __shfl_xor(m2, 16, 64));
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
        for (int i = 0; i < V; ++i) key[i] = kept ? key[i] : 0u;
    }

    int mine = 0;   // lane j: the place of the token's j-th expert
    if constexpr (V <= 8) {
        uint64_t pos = 0;   // the sorted keys' places, 8 bits each
        int p[V];
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = i;
        // exchanges of neighbours only, and only of unequal ones: equal keys keep their order
#pragma unroll
        for (int r = 0; r < V; ++r) {
#pragma unroll
            for (int i = r & 1; i + 1 < V; i += 2) {
                const uint32_t ki = key[i], kj = key[i + 1];
                const int pi = p[i], pj = p[i + 1];
                const bool up = ki < kj;
                key[i] = umax(ki, kj), key[i + 1] = umin(ki, kj);
                p[i] = up ? pj : pi, p[i + 1] = up ? pi : pj;
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) pos |= (uint64_t)p[i] << (8 * i);
        for (int j = 0; j < a.k; ++j) {
            const uint32_t best = wave_max(key[0]);
            const int owner = __builtin_ctzll(__ballot(key[0] == best));
            const int place = owner * V + (__builtin_amdgcn_readlane((int)(uint32_t)pos, owner) & 0xFF);
            mine = lane == j ? place : mine;
            const bool own = lane == owner;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const uint32_t here = key[i], next = i + 1 < V ? key[i + 1] : 0u;
                key[i] = own ? next : here;
            }
            if constexpr (V <= 4) pos = own ? (uint32_t)pos >> 8 : (uint32_t)pos;
            else pos = own ? pos >> 8 : pos;
        }
    } else {
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
            const int place = owner * V + __builtin_amdgcn_readlane(pos, owner);
            mine = lane == j ? place : mine;
        }
    }

    // (LDS accesses of a wave run in order; the fence keeps the compiler's order)
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    float w = lane < a.k ? reinterpret_cast<const float *>(rows[wave])[mine] : 0.0f;
    const int from = mine / V;   // the lane that holds it
    const int expert = (from >> a.lane_shift) * a.per + (from & (lanes - 1)) * V + mine % V;
    if (a.renormalize) {
        const float sum = wave_sum(w);
        w = sum != 0.0f ? w / sum : 0.0f;   // (a token none of whose experts has a score has weights 0)
    }
    if (lane < a.k) {
        a.weights[t * a.k + lane] = w * a.scale;
        a.experts[t * a.k + lane] = expert;
    }
}

// Many tokens: 16 lanes (a team) to a token, four tokens to a wave. The steps are those of
// route_kernel, each of them for four tokens at once and over 16 lanes instead of 64. Of a lane's
// up to 16 experts every four are sorted; a step takes the largest of their first ones. A team's
// first lane among those at the maximum is the lowest set bit of its 16 in a ballot. Bound by its
// operations too (237 a token; a third of them the scores): 16384 tokens' 256 experts 10.4 us
// against 13.0 with a wave to a token, of which 3 are the launch.
__device__ __forceinline__ uint64_t first_of_teams(uint64_t m) {   // (no 16 bits of m are all clear)
    return m & (~m + 0x0001000100010001ull);
}

template <int V, int BF16, int SOFTMAX, int QUADS>
__global__ __launch_bounds__(64 * kWaves) void route_teams_kernel(RouteArgs a) {
    constexpr int Q = V / 4;
    __shared__ u32x4 keys[kWaves][64 * Q];
    __shared__ uint32_t places[kWaves][64 * Q], picks[kWaves][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t0 = ((int64_t)blockIdx.x * kWaves + wave) * 4;
    if (t0 >= a.T) return;
    const int tl = lane & 15;
    const bool there = t0 + (lane >> 4) < a.T;
    const int64_t t = there ? t0 + (lane >> 4) : t0;   // (teams without a token repeat the first)
    const int lanes = 1 << a.lane_shift;
    const int group = tl >> a.lane_shift;
    const int at = (tl & (lanes - 1)) * V;
    const int n = group < a.groups ? max(min(a.per - at, V), 0) : 0;
    const int e0 = group * a.per + at;
    const int64_t row = t * a.E;

    float x[V], s[V], bias[V], top = 0.0f, total = 1.0f;
    if constexpr (QUADS) load_quads<V, BF16>(a.logits, row, e0, n, x);
    else load_row<V, BF16, 0>(a.logits, row, e0, n, a.E, x);
#pragma unroll
    for (int i = 0; i < V; ++i) bias[i] = 0.0f;
    if (a.bias) {
        if constexpr (QUADS) load_quads<V, 0>(a.bias, 0, e0, n, bias);
        else load_row<V, 0, 0>(a.bias, 0, e0, n, a.E, bias);
    }
    if constexpr (SOFTMAX) {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = n > (QUADS ? i & ~3 : i) ? x[i] : -__builtin_inff();
    }
    scores<V, SOFTMAX, 1>(x, s, top, total);
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const uint32_t k = key_of(s[i] + bias[i]);
        key[i] = n > (QUADS ? i & ~3 : i) ? k : 0u;
    }

    if (a.groups > 1) {
        uint32_t m1 = key[0], m2 = 0;
#pragma unroll
        for (int i = 1; i < V; ++i) merge2(m1, m2, key[i], 0);
        if (lanes > 1) merge2(m1, m2, dpp<kXor1>(m1), dpp<kXor1>(m2));
        if (lanes > 2) merge2(m1, m2, dpp<kXor2>(m1), dpp<kXor2>(m2));
        if (lanes > 4) merge2(m1, m2, dpp<kMirror8>(m1), dpp<kMirror8>(m2));
        uint32_t value = m1;
        if (a.group_top2 && m2) value = key_of(of_key(m1) + of_key(m2));
        uint64_t kept = 0;
        for (int r = 0; r < a.topk_groups; ++r) {
            const uint32_t best = team_max(value);
            const uint64_t first = first_of_teams(__ballot(value == best));
            const uint64_t block = (first << lanes) - first;   // all lanes of those groups
            kept |= block;
            value = __builtin_amdgcn_inverse_ballot_w64(block) ? 0u : value;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = __builtin_amdgcn_inverse_ballot_w64(kept) ? key[i] : 0u;
    }

    // Quad q's first key stays in a register, the others and a 0 go to LDS, from where the next one
    // comes when the first is taken. next[q]: where it lies, which also says which key the first is:
    // quarters of these addresses index the keys' places in the lane. (The quads are exchanged
    // among a lane's by its number, against bank conflicts.)
    uint32_t head[Q], next[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        uint32_t p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = 4 * q + i;
        // exchanges of neighbours only, and only of unequal ones: equal keys keep their order
#pragma unroll
        for (int r = 0; r < 4; ++r) {
#pragma unroll
            for (int i = r & 1; i + 1 < 4; i += 2) {
                const uint32_t ki = key[4 * q + i], kj = key[4 * q + i + 1], pi = p[i], pj = p[i + 1];
                const bool up = ki < kj;
                key[4 * q + i] = umax(ki, kj), key[4 * q + i + 1] = umin(ki, kj);
                p[i] = up ? pj : pi, p[i + 1] = up ? pi : pj;
            }
        }
        const int at_q = lane * Q + (Q == 3 ? q : q ^ (lane / (16 / Q) & (Q - 1)));
        keys[wave][at_q] = u32x4{key[4 * q + 1], key[4 * q + 2], key[4 * q + 3], 0u};
        places[wave][at_q] = p[0] | p[1] << 8 | p[2] << 16 | p[3] << 24;
        head[q] = key[4 * q];
        next[q] = 16 * at_q;
    }
    for (int j = 0; j < a.k; ++j) {
        uint32_t most = head[0];
#pragma unroll
        for (int q = 1; q < Q; ++q) most = umax(most, head[q]);
        const uint32_t best = team_max(most);
        const uint64_t own = first_of_teams(__ballot(most == best));
        uint64_t hits[Q], open = own;   // the lanes whose quad q it is, the first with that key
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            hits[q] = q + 1 < Q ? open & __ballot(head[q] == best) : open;
            open &= ~hits[q];
        }
        uint32_t following = 0;
        if (__builtin_amdgcn_inverse_ballot_w64(own)) {
            uint32_t from = next[0];
#pragma unroll
            for (int q = 1; q < Q; ++q) from = __builtin_amdgcn_inverse_ballot_w64(hits[q]) ? next[q] : from;
            following = *reinterpret_cast<const uint32_t *>(reinterpret_cast<const uint8_t *>(keys[wave]) + from);
            picks[wave][(lane & 48) + j] = from;
        }
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const bool hit = __builtin_amdgcn_inverse_ballot_w64(hits[q]);
            head[q] = hit ? following : head[q];
            next[q] += hit ? 4 : 0;
        }
    }

    // (LDS accesses of a wave run in order; the fence keeps the compiler's order)
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const uint32_t pick = tl < a.k ? picks[wave][lane] : 0u;
    const int from = pick / (16 * Q) & 15, place = reinterpret_cast<const uint8_t *>(places[wave])[pick / 4];
    const int expert = (from >> a.lane_shift) * a.per + (from & (lanes - 1)) * V + place;
    // its score again, from its logit: cheaper than keeping every score at hand
    float w = tl < a.k ? score_of<SOFTMAX>(load_logit<BF16>(a.logits, row + expert), top, total) : 0.0f;
    if (a.renormalize) {
        const float sum = team_sum(w);
        w = sum != 0.0f ? w / sum : 0.0f;
    }
    if (there && tl < a.k) {
        a.weights[t * a.k + tl] = w * a.scale;
        a.experts[t * a.k + tl] = expert;
    }
}

// Scores whose sum is less are scaled up by kUp, so that neither they nor quotients by their sum leave
// fp32's range
constexpr float kSmallSum = 0x1p-64f, kUp = 0x1p64f;

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
// ds passes fp32's range where S is about as small as its smallest numbers: there the scores are
// scaled up by a power of two and ds is that much smaller, which leaves the products as they are.
// The row of ds goes through LDS, from the k selected experts' lanes to the experts' lanes. Bound
// by its operations with few tokens to a chip's worth of waves (softmax, 16384 tokens' 256 experts
// 10.2 us), in teams by memory (65536 tokens 27 us, 5.1 TB/s; 22 where the caches still hold the logits).
template <int V, int BF16, int SOFTMAX, int FULL>
__global__ __launch_bounds__(64 * kWaves) void route_grad_kernel(RouteGradArgs a) {
    typedef float piece __attribute__((ext_vector_type(V)));
    __shared__ piece rows[kWaves][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t = (int64_t)blockIdx.x * kWaves + wave;
    if (t >= a.T) return;
    const int e0 = lane * V, n = max(min(a.E - e0, V), 0);
    const int64_t row = t * a.E;

    const int e = lane < a.k ? a.experts[t * a.k + lane] : -1;
    const bool there = e >= 0 && e < a.E;
    const float dw = there ? a.dweights[t * a.k + lane] : 0.0f;
    const float xe = load_logit<BF16>(a.logits, row + (there ? e : 0));
    float x[V], p[V], top = 0.0f, total = 1.0f;
    if constexpr (SOFTMAX) {
        load_row<V, BF16, FULL>(a.logits, row, e0, n, a.E, x);
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = has<FULL>(i, n) ? x[i] : -__builtin_inff();
        scores<V, 1>(x, p, top, total);
    }
    piece zero;
#pragma unroll
    for (int i = 0; i < V; ++i) zero[i] = 0.0f;
    rows[wave][lane] = zero;

    const float s = there ? score_of<SOFTMAX>(xe, top, total) : 0.0f;
    float d = dw * a.scale, z = s;   // z: the score, scaled up if need be
    bool small = false;
    if (a.renormalize) {
        float sum = wave_sum(s);
        small = sum < kSmallSum;
        z = small ? s * kUp : s;
        sum = small ? sum * kUp : sum;
        const float dot = wave_sum(d * z);
        d = there && sum != 0.0f ? (d - dot / sum) / sum : 0.0f;
    }
    float all = SOFTMAX ? wave_sum(d * z) : 0.0f;
    if constexpr (SOFTMAX) {
        if (__any(small)) {
#pragma unroll
            for (int i = 0; i < V; ++i) p[i] = small ? p[i] * kUp : p[i];
            all = small ? all / kUp : all;
        }
    } else {
        d *= z * (1.0f - s);
    }
    // (LDS accesses of a wave run in order; the fences keep the compiler's order)
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (there) reinterpret_cast<float *>(rows[wave])[e] = d;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");

    piece g = rows[wave][lane];
    if constexpr (SOFTMAX) {
#pragma unroll
        for (int i = 0; i < V; ++i) g[i] = p[i] * (g[i] - all);
    }
    if constexpr (BF16) {
        typedef uint16_t half_piece __attribute__((ext_vector_type(V)));
        half_piece h;
#pragma unroll
        for (int i = 0; i < V; ++i) h[i] = (uint16_t)pack_bf16x2(g[i], 0.0f);
        uint16_t *dst = reinterpret_cast<uint16_t *>(a.dlogits) + row + e0;
        if constexpr (FULL) {
            if (n > 0) *reinterpret_cast<half_piece *>(dst) = h;
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i < n) dst[i] = h[i];
        }
    } else {
        float *dst = reinterpret_cast<float *>(a.dlogits) + row + e0;
        if constexpr (FULL) {
            if (n > 0) *reinterpret_cast<piece *>(dst) = g;
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i < n) dst[i] = g[i];
        }
    }
}

// n of 4 consecutive elements at i. QUADS: all or none, aligned.
template <int BF16, int QUADS>
__device__ __forceinline__ void store_quad(void *p, int64_t i, int n, f32x4 g) {
    if constexpr (BF16) {
        typedef uint16_t piece __attribute__((ext_vector_type(4)));
        piece h;
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = (uint16_t)pack_bf16x2(g[j], 0.0f);
        uint16_t *dst = reinterpret_cast<uint16_t *>(p) + i;
        if constexpr (QUADS) {
            if (n > 0) *reinterpret_cast<piece *>(dst) = h;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < n) dst[j] = h[j];
        }
    } else {
        float *dst = reinterpret_cast<float *>(p) + i;
        if constexpr (QUADS) {
            if (n > 0) *reinterpret_cast<f32x4 *>(dst) = g;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < n) dst[j] = g[j];
        }
    }
}

// Many tokens: 16 lanes to a token. Quad q of lane l is experts 64 q + 4 l and on, so that a
// team's accesses are contiguous.
template <int Q, int BF16, int SOFTMAX, int QUADS>
__global__ __launch_bounds__(64 * kWaves) void route_grad_teams_kernel(RouteGradArgs a) {
    constexpr int V = 4 * Q;
    __shared__ f32x4 rows[kWaves][4][16 * Q];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t0 = ((int64_t)blockIdx.x * kWaves + wave) * 4;
    if (t0 >= a.T) return;
    const int tl = lane & 15, team = lane >> 4;
    const bool real = t0 + team < a.T;
    const int64_t t = real ? t0 + team : t0;   // (teams without a token repeat the first, and store nothing)
    const int64_t row = t * a.E;

    const int e = tl < a.k ? a.experts[t * a.k + tl] : -1;
    const bool there = e >= 0 && e < a.E;
    const float dw = there ? a.dweights[t * a.k + tl] : 0.0f;
    const float xe = load_logit<BF16>(a.logits, row + (there ? e : 0));
    float p[V], top = 0.0f, total = 1.0f;
    if constexpr (SOFTMAX) {
        float x[V];
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int first = 64 * q + 4 * tl;
            float quad[4];
            load_row<4, BF16, QUADS>(a.logits, row, first, a.E - first, a.E, quad);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[4 * q + i] = first + i < a.E ? quad[i] : -__builtin_inff();
        }
        scores<V, 1, 1>(x, p, top, total);
    }
#pragma unroll
    for (int q = 0; q < Q; ++q) rows[wave][team][16 * q + tl] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    const float s = there ? score_of<SOFTMAX>(xe, top, total) : 0.0f;
    float d = dw * a.scale, z = s;   // z: the score, scaled up if need be
    bool small = false;
    if (a.renormalize) {
        float sum = team_sum(s);
        small = sum < kSmallSum;
        z = small ? s * kUp : s;
        sum = small ? sum * kUp : sum;
        const float dot = team_sum(d * z);
        d = there && sum != 0.0f ? (d - dot / sum) / sum : 0.0f;
    }
    float all = SOFTMAX ? team_sum(d * z) : 0.0f;
    if constexpr (SOFTMAX) {
        if (__any(small)) {
#pragma unroll
            for (int i = 0; i < V; ++i) p[i] = small ? p[i] * kUp : p[i];
            all = small ? all / kUp : all;
        }
    } else {
        d *= z * (1.0f - s);
    }
    // (LDS accesses of a wave run in order; the fences keep the compiler's order)
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (there) reinterpret_cast<float *>(rows[wave][team])[e] = d;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");

#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int first = 64 * q + 4 * tl;
        f32x4 g = rows[wave][team][16 * q + tl];
        if constexpr (SOFTMAX) {
#pragma unroll
            for (int i = 0; i < 4; ++i) g[i] = p[4 * q + i] * (g[i] - all);
        }
        if (!real) continue;
        store_quad<BF16, QUADS>(a.dlogits, row + first, a.E - first, g);
    }
}

template <int V, int BF16, int SOFTMAX, int TEAM>
void route_f(const RouteArgs &a, bool full, dim3 grid, hipStream_t st) {
    const dim3 block(64 * kWaves);
    if constexpr (TEAM) {
        if (full) route_teams_kernel<V, BF16, SOFTMAX, 1><<<grid, block, 0, st>>>(a);
        else route_teams_kernel<V, BF16, SOFTMAX, 0><<<grid, block, 0, st>>>(a);
        return;
    }
    if constexpr (V > 1) {
        if (full) {
            route_kernel<V, BF16, SOFTMAX, 1><<<grid, block, 0, st>>>(a);
            return;
        }
    }
    route_kernel<V, BF16, SOFTMAX, 0><<<grid, block, 0, st>>>(a);
}

template <int V, int BF16, int SOFTMAX, int TEAM>
void route_grad_f(const RouteGradArgs &a, bool full, dim3 grid, hipStream_t st) {
    const dim3 block(64 * kWaves);
    if constexpr (TEAM) {
        if (full) route_grad_teams_kernel<V / 4, BF16, SOFTMAX, 1><<<grid, block, 0, st>>>(a);
        else route_grad_teams_kernel<V / 4, BF16, SOFTMAX, 0><<<grid, block, 0, st>>>(a);
        return;
    }
    if constexpr (V > 1) {
        if (full) {
            route_grad_kernel<V, BF16, SOFTMAX, 1><<<grid, block, 0, st>>>(a);
            return;
        }
    }
    route_grad_kernel<V, BF16, SOFTMAX, 0><<<grid, block, 0, st>>>(a);
}

// Whether every lane's V elements of a row come in one access: rows and groups are whole
// numbers of V elements, and the buffers aligned to them (16 bytes at most are needed).
bool whole(int V, int per, bool bf16, const void *p, const void *q) {
    const uintptr_t bytes = (uintptr_t)V * (bf16 ? 2 : 4), mask = (bytes < 16 ? bytes : 16) - 1;
    return per % V == 0 && ((reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(q)) & mask) == 0;
}

template <int V, int TEAM>
void route_v(const RouteArgs &a, bool bf16, bool softmax, dim3 grid, hipStream_t st) {
    constexpr int W = TEAM ? 4 : V;
    const bool full = whole(W, a.per, bf16, a.logits, nullptr) && whole(W, a.per, false, a.bias, nullptr);
    if (bf16) {
        if (softmax) route_f<V, 1, 1, TEAM>(a, full, grid, st);
        else route_f<V, 1, 0, TEAM>(a, full, grid, st);
    } else {
        if (softmax) route_f<V, 0, 1, TEAM>(a, full, grid, st);
        else route_f<V, 0, 0, TEAM>(a, full, grid, st);
    }
}

template <int V, int TEAM>
void route_grad_v(const RouteGradArgs &a, bool bf16, bool softmax, dim3 grid, hipStream_t st) {
    const bool full = whole(TEAM ? 4 : V, a.E, bf16, a.logits, a.dlogits);
    if (bf16) {
        if (softmax) route_grad_f<V, 1, 1, TEAM>(a, full, grid, st);
        else route_grad_f<V, 1, 0, TEAM>(a, full, grid, st);
    } else {
        if (softmax) route_grad_f<V, 0, 1, TEAM>(a, full, grid, st);
        else route_grad_f<V, 0, 0, TEAM>(a, full, grid, st);
    }
}

}  // namespace

hipError_t launch_moe_route(const void *logits, bool bf16, const float *bias, float *weights, int32_t *experts,
                            int64_t T, int E, int k, int groups, int topk_groups, bool softmax, bool group_top2,
                            bool renormalize, float scale, hipStream_t stream) {
    RouteArgs a{logits, bias, weights, experts, T, E, k, groups, topk_groups, E / groups, 6, group_top2, renormalize,
                scale};
    for (int g = 1; g < groups; g <<= 1) --a.lane_shift;
    // Teams from the number of tokens on at which their waves fill the chip. A wave to a token
    // against teams, us, three sets of inputs in turn: 256 experts (16 a lane) at 4096 / 8192 / 16384 / 65536
    // tokens 5.5 / 7.7 / 13.0 / 41 against 5.6 / 6.7 / 10.4 / 27; 64 experts (4 a lane) at 2048 / 8192 / 65536
    // 4.2 / 5.6 / 27 against 4.3 / 4.8 / 12.
    const int v4 = ((a.per - 1) >> max(a.lane_shift - 2, 0)) + 1, quads = (v4 + 3) / 4;   // of a lane of 16
    if (T >= 2048 * quads && k <= 16 && groups <= 16 && quads <= 4) {
        a.lane_shift -= 2;
        const dim3 teams((unsigned)((T + 4 * kWaves - 1) / (4 * kWaves)));
        if (quads == 1) route_v<4, 1>(a, bf16, softmax, teams, stream);
        else if (quads == 2) route_v<8, 1>(a, bf16, softmax, teams, stream);
        else if (quads == 3) route_v<12, 1>(a, bf16, softmax, teams, stream);
        else route_v<16, 1>(a, bf16, softmax, teams, stream);
        return hipGetLastError();
    }
    const int v = ((a.per - 1) >> a.lane_shift) + 1;   // experts per lane
    const dim3 grid((unsigned)((T + kWaves - 1) / kWaves));
    if (v <= 1) route_v<1, 0>(a, bf16, softmax, grid, stream);
    else if (v <= 2) route_v<2, 0>(a, bf16, softmax, grid, stream);
    else if (v <= 4) route_v<4, 0>(a, bf16, softmax, grid, stream);
    else if (v <= 8) route_v<8, 0>(a, bf16, softmax, grid, stream);
    else if (v <= 16) route_v<16, 0>(a, bf16, softmax, grid, stream);
    else if (v <= 32) route_v<32, 0>(a, bf16, softmax, grid, stream);
    else return hipErrorInvalidValue;
    return hipGetLastError();
}

hipError_t launch_moe_route_backward(const float *dweights, const void *logits, bool bf16, const int32_t *experts,
                                     void *dlogits, int64_t T, int E, int k, bool softmax, bool renormalize,
                                     float scale, hipStream_t stream) {
    const RouteGradArgs a{dweights, logits, experts, dlogits, T, E, k, renormalize, scale};
    const dim3 grid((unsigned)((T + kWaves - 1) / kWaves));
    // Teams or a wave to a token, us, three sets of inputs in turn: softmax, 256 experts at 4096 / 8192 / 65536
    // tokens 4.7 / 5.6 / 27 against 4.7 / 6.3 / 33, 64 experts at 8192 / 65536 4.9 / 9.3 against 4.9 / 22. (Rows
    // that are no whole quads are loaded by elements: 255 experts, 16384 tokens 12.5 against 11.1.)
    if (T >= 4096 && k <= 16 && E <= (E % 4 == 0 ? 256 : 192)) {
        const dim3 teams((unsigned)((T + 4 * kWaves - 1) / (4 * kWaves)));
        if (E <= 64) route_grad_v<4, 1>(a, bf16, softmax, teams, stream);
        else if (E <= 128) route_grad_v<8, 1>(a, bf16, softmax, teams, stream);
        else if (E <= 192) route_grad_v<12, 1>(a, bf16, softmax, teams, stream);
        else route_grad_v<16, 1>(a, bf16, softmax, teams, stream);
        return hipGetLastError();
    }
    if (E <= 64) route_grad_v<1, 0>(a, bf16, softmax, grid, stream);
    else if (E <= 128) route_grad_v<2, 0>(a, bf16, softmax, grid, stream);
    else if (E <= 256) route_grad_v<4, 0>(a, bf16, softmax, grid, stream);
    else if (E <= 512) route_grad_v<8, 0>(a, bf16, softmax, grid, stream);
    else if (E <= 1024) route_grad_v<16, 0>(a, bf16, softmax, grid, stream);
    else return hipErrorInvalidValue;
    return hipGetLastError();
}

}  // namespace fp8q
