// norm.hip -- the norms before and after a block, with the block's gate and the residual, in one pass
// over the rows, and their gradient.
//
//     n = y, or with `post` y * q * post, q = 1 / sqrt(mean(y^2) + eps)
//     t = scale * x + gate * n                       gate: one per channel, per element, or 1
//     z = t * r * weight, r = 1 / sqrt(mean(t^2) + eps)
//
// and from dt (of t besides z) and dz, with th = t * r and yh = y * q:
//
//     d = dt + r * (dz * weight - th * mean(dz * weight * th)),  dx = scale * d,  dweight = sum dz * th
//     dn = d * gate,  dgate = d * n (summed over the rows for one per channel),  dpost = sum dn * yh
//     dy = dn, or with `post` q * (dn * post - yh * mean(dn * post * yh))
//
// Bound by memory: four rows of H elements a token, six for the gradient. So a row is read once, into
// registers, NT threads to a row and NV pieces of 8 elements a thread, and a workgroup walks many rows:
// the per-channel vectors stay in registers too, up to 8192 channels (read again for every row they would be
// more bytes than the rows themselves, if from the caches), the next row's loads are on their way while a row is
// reduced, and the gradient's sums over the rows are carried in registers. Squares, sums and every step are fp32; t
// enters the second norm before its rounding. Outputs round once. The order of every sum is fixed.
// 16384 x 7168 bf16 177 us, 5.3 TB/s (a copy of 1 GB: 5.15); the gradient of 4096 x 7168 94 us, 3.7 TB/s, of
// 16384 x 2048 82 us, 4.9 TB/s. One row of 7168 takes 4 us on the device, most of it two dependent sums. Rows above 8192
// outgrow the gradient's registers: their statistics and the rest are two kernels.
#include <fp8q.h>

#include "device_common.h"
#include "launch.h"

namespace fp8q {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
// rows of any length: pieces lie at the alignment of an element
typedef u32x4 __attribute__((aligned(2))) u32x4_any;

struct NormArgs {
    const void *x, *y;          // the gradient: x is t
    const void *dt, *dz;        // gradient only; dt may be null
    const float *weight, *post; // [H] or null
    const float *gate;          // [H] or null
    const void *gates;          // [T, H] or null (at most one of gate, gates)
    void *t, *z;                // the gradient: dx, dy
    void *dgates;               // gradient: [T, H], or null
    float *sums[3];             // gradient: dweight, dpost, dgate, each [partials][H] at `pitch`
    int64_t pitch;
    int64_t T;
    int H;
    float scale, eps;
};

// 8 elements as they come from memory
template <int BF16>
struct Raw {
    u32x4 v[BF16 ? 1 : 2];
    __device__ __forceinline__ float at(int i) const {
        if constexpr (BF16) return i & 1 ? bf16hi_to_f32(v[0][i / 2]) : bf16lo_to_f32(v[0][i / 2]);
        else return __uint_as_float(v[i / 4][i % 4]);
    }
};

// Piece p of a row of H >= 8 elements, in two steps: a load that needs no branch (from the row's last 8
// elements where the piece is short or past the end), and, once it is there, what lies before the piece shifted out
// and zeros put past the row's end. (Done at once, the wait for the load would come before the work that is to hide it.)
template <int BF16>
__device__ __forceinline__ Raw<BF16> load8(const void *base, int64_t row, int p, int H) {
    const uint32_t off = 8 * p + 8 <= H ? 8 * p : H - 8;
    const char *from = static_cast<const char *>(base) + row * H * (BF16 ? 2 : 4);
    Raw<BF16> r;
#pragma unroll
    for (int h = 0; h < (BF16 ? 1 : 2); ++h)
        r.v[h] = *reinterpret_cast<const u32x4_any *>(from + (uint32_t)(off * (BF16 ? 2 : 4) + 16 * h));
    return r;
}
template <int BF16>
__device__ __forceinline__ Raw<BF16> settle(Raw<BF16> r, int p, int H) {
    constexpr int N = BF16 ? 1 : 2;
    const int s = 8 * p + 8 - H;   // elements past the end
    if (s > 0) {
        uint32_t u[4 * N];
#pragma unroll
        for (int i = 0; i < 4 * N; ++i) u[i] = s >= 8 ? 0 : r.v[i / 4][i % 4];
#pragma unroll
        for (int bit = 4; bit; bit >>= 1) {
            const int words = BF16 ? bit / 2 : bit;   // (half a word last, of bf16)
#pragma unroll
            for (int i = 0; i < 4 * N; ++i) {
                const uint32_t up = words ? (i + words < 4 * N ? u[i + words] : 0)
                                          : u[i] >> 16 | (i + 1 < 4 * N ? u[i + 1] << 16 : 0);
                u[i] = s & bit ? up : u[i];
            }
        }
#pragma unroll
        for (int i = 0; i < 4 * N; ++i) r.v[i / 4][i % 4] = u[i];
    }
    return r;
}

template <int BF16>
__device__ __forceinline__ void store8(void *base, int64_t row, int p, int H, const float (&v)[8]) {
    const int left = H - 8 * p;
    if (left <= 0) return;
    if constexpr (BF16) {
        uint16_t *q = reinterpret_cast<uint16_t *>(static_cast<char *>(base) + row * H * 2 + (uint32_t)(16 * p));
        const u32x4 u = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                         pack_bf16x2(v[6], v[7])};
        if (left >= 8) {
            *reinterpret_cast<u32x4_any *>(q) = u;
        } else {
#pragma unroll
            for (int i = 0; i < 7; ++i)
                if (i < left) q[i] = (uint16_t)(u[i / 2] >> (16 * (i & 1)));
        }
    } else {
        float *q = reinterpret_cast<float *>(static_cast<char *>(base) + row * H * 4 + (uint32_t)(32 * p));
        if (left >= 8) {
            *reinterpret_cast<u32x4_any *>(q) = __builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]});
            *reinterpret_cast<u32x4_any *>(q + 4) = __builtin_bit_cast(u32x4, f32x4{v[4], v[5], v[6], v[7]});
        } else {
#pragma unroll
            for (int i = 0; i < 7; ++i)
                if (i < left) q[i] = v[i];
        }
    }
}

// A per-channel vector's pieces of this thread, ones where there is none: kept in registers, or read
// again for every row where a row takes too many of them
template <int NT, int NV, bool KEEP>
struct Channels {
    Raw<0> kept[KEEP ? NV : 1];
    const float *v;
    int tid, H;
    __device__ __forceinline__ Channels(const float *v_, int tid_, int H_) : v(v_), tid(tid_), H(H_) {
        if constexpr (KEEP) {
#pragma unroll
            for (int i = 0; i < NV; ++i) kept[i] = read(i);
        }
    }
    __device__ __forceinline__ Raw<0> read(int i) const {
        if (v) return settle<0>(load8<0>(v, 0, tid + i * NT, H), tid + i * NT, H);
        Raw<0> r;
        r.v[0] = r.v[1] = u32x4{0x3F800000u, 0x3F800000u, 0x3F800000u, 0x3F800000u};
        return r;
    }
    __device__ __forceinline__ Raw<0> operator()(int i) const {
        if constexpr (KEEP) return kept[i];
        else return read(i);
    }
};

// The sum over a wave, in every lane: 16 lanes by DPP moves, then the four 16s
template <int CTRL>
__device__ __forceinline__ float moved(float v) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ float lane_of(float v, int lane) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), lane));
}
__device__ __forceinline__ float wave_sum(float v) {
    v += moved<0xB1>(v);    // quad_perm [1,0,3,2]
    v += moved<0x4E>(v);    // quad_perm [2,3,0,1]
    v += moved<0x141>(v);   // row_half_mirror
    v += moved<0x140>(v);   // row_mirror
    return (lane_of(v, 0) + lane_of(v, 16)) + (lane_of(v, 32) + lane_of(v, 48));
}

// Sums of N values over the NT threads of a row, the same bits in all of them. `turn` alternates: the
// values of one call stay readable until every thread is past the barrier of the next.
template <int NT, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*part)[3][NT / 64], int &turn) {
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] = wave_sum(v[n]);
    if constexpr (NT > 64) {
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int n = 0; n < N; ++n) part[turn][n][threadIdx.x >> 6] = v[n];
        }
        // (a barrier that waits for LDS, not for the next row's loads)
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (0 << 8) | (3 << 14));
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
#pragma unroll
        for (int n = 0; n < N; ++n) {
            v[n] = part[turn][n][0];
#pragma unroll
            for (int w = 1; w < NT / 64; ++w) v[n] += part[turn][n][w];
        }
        turn ^= 1;
    }
}

// NT threads to a row: a wave (four rows a workgroup) or a workgroup
template <int NT>
constexpr int rows_of() { return NT == 64 ? 4 : 1; }

// GATES: the gate is one per element
template <int BF16, int NT, int NV, int GATES>
__global__ __launch_bounds__(NT * rows_of<NT>()) void residual_norm_kernel(NormArgs g) {
    constexpr int ROWS = rows_of<NT>();
    // The channels in registers; of rows above 8192, whose next row's loads already fill those, read again for each row.
    // us, read / held: bf16 4096 x 12288 with a gate per element 100 / 117, fp32 289 / 309; without 93 / 93, 229 / 229
    constexpr bool HELD = NV == 1;
    __shared__ float part[2][3][NT / 64];
    const int tid = threadIdx.x % NT, H = g.H;
    const int64_t step = (int64_t)gridDim.x * ROWS;
    int64_t row = (int64_t)blockIdx.x * ROWS + __builtin_amdgcn_readfirstlane(threadIdx.x / NT);
    const float inv = 1.0f / (float)H;
    int turn = 0;

    Raw<BF16> x[NV], y[NV], gt[NV];
    auto load = [&](int64_t m) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            x[i] = load8<BF16>(g.x, m, tid + i * NT, H);
            if (g.y) y[i] = load8<BF16>(g.y, m, tid + i * NT, H);
            if constexpr (GATES) gt[i] = load8<BF16>(g.gates, m, tid + i * NT, H);
        }
    };
    if (row < g.T) load(row);
    const Channels<NT, NV, HELD> weight(g.weight, tid, H), post(g.post, tid, H), gate(g.gate, tid, H);
    for (; row < g.T; row += step) {
        float t[NV][8], n[NV][8];
        Raw<BF16> gates[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int p = tid + i * NT;
            if constexpr (GATES) gates[i] = settle(gt[i], p, H);
            const Raw<BF16> xs = settle(x[i], p, H);
            Raw<BF16> ys;
            if (g.y) ys = settle(y[i], p, H);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                t[i][e] = g.scale * xs.at(e);
                n[i][e] = g.y ? ys.at(e) : 0.0f;
            }
        }
        if (row + step < g.T) load(row + step);
        if (g.y) {
            float q = 1.0f;
            if (g.post) {
                float s[1] = {0.0f};
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int e = 0; e < 8; ++e) s[0] = __builtin_fmaf(n[i][e], n[i][e], s[0]);
                row_sums<NT>(s, part, turn);
                q = 1.0f / __builtin_sqrtf(s[0] * inv + g.eps);
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const Raw<0> p = post(i), c = gate(i);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    t[i][e] = __builtin_fmaf(GATES ? gates[i].at(e) : c.at(e), n[i][e] * q * p.at(e), t[i][e]);
            }
        }
        if (g.t) {
#pragma unroll
            for (int i = 0; i < NV; ++i) store8<BF16>(g.t, row, tid + i * NT, H, t[i]);
        }
        if (g.weight) {
            float s[1] = {0.0f};
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) s[0] = __builtin_fmaf(t[i][e], t[i][e], s[0]);   // (0 past the row's end)
            row_sums<NT>(s, part, turn);
            const float r = 1.0f / __builtin_sqrtf(s[0] * inv + g.eps);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const Raw<0> w = weight(i);
#pragma unroll
                for (int e = 0; e < 8; ++e) t[i][e] = t[i][e] * r * w.at(e);
                store8<BF16>(g.z, row, tid + i * NT, H, t[i]);
            }
        }
    }
}

// The same in LDS, for the gradient, whose sums over the rows take the registers: 16 bytes of each of a
// wave's lanes side by side, which meets no bank conflict.
template <int NT, int NV>
struct SharedChannels {
    f32x4 *at;
    int tid;
    static constexpr int SIZE = 2 * NT * NV;
    __device__ __forceinline__ SharedChannels(f32x4 *lds, const float *v, int tid_, int H) : at(lds), tid(tid_) {
        // (a workgroup's waves write the same where each has a row)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Raw<0> r = Channels<NT, NV, false>(v, tid, H).read(i);
#pragma unroll
            for (int h = 0; h < 2; ++h) at[(2 * i + h) * NT + tid] = __builtin_bit_cast(f32x4, r.v[h]);
        }
    }
    __device__ __forceinline__ f32x4 operator()(int i, int h) const { return at[(2 * i + h) * NT + tid]; }   // half h of piece i
};

// keeps the compiler from holding what it has computed from v: that is computed again from v instead
template <int BF16>
__device__ __forceinline__ void forget(Raw<BF16> &v) {
#pragma unroll
    for (int h = 0; h < (BF16 ? 1 : 2); ++h) asm volatile("" : "+v"(v.v[h]));
}

// What the gradient takes from row m, piece tid + i NT of it; what is not there counts as zeros
template <int BF16, int NT, int GATES>
struct GradInputs {
    struct Piece {
        Raw<BF16> t, dz, dt, y, gate;
    };
    const NormArgs &g;
    int tid;
    bool need_y;
    __device__ __forceinline__ GradInputs(const NormArgs &g_, int tid_)
        : g(g_), tid(tid_), need_y(g_.y && (g_.post || g_.sums[2] || GATES)) {}
    __device__ __forceinline__ Piece read(int64_t m, int i) const {
        Piece p;
#pragma unroll
        for (int h = 0; h < (BF16 ? 1 : 2); ++h)
            p.t.v[h] = p.dz.v[h] = p.dt.v[h] = p.y.v[h] = p.gate.v[h] = u32x4{0, 0, 0, 0};
        if (g.weight) {
            p.t = load8<BF16>(g.x, m, tid + i * NT, g.H);
            p.dz = load8<BF16>(g.dz, m, tid + i * NT, g.H);
        }
        if (g.dt) p.dt = load8<BF16>(g.dt, m, tid + i * NT, g.H);
        if (need_y) p.y = load8<BF16>(g.y, m, tid + i * NT, g.H);
        if constexpr (GATES) p.gate = load8<BF16>(g.gates, m, tid + i * NT, g.H);
        return p;
    }
    __device__ __forceinline__ Piece settled(Piece p, int i) const {
        const int at = tid + i * NT;
        p.t = settle(p.t, at, g.H), p.dz = settle(p.dz, at, g.H), p.dt = settle(p.dt, at, g.H), p.y = settle(p.y, at, g.H);
        if constexpr (GATES) p.gate = settle(p.gate, at, g.H);
        return p;
    }
};

// The gradient. The sums over the rows leave as one partial row per workgroup, which a second kernel
// adds up (with one workgroup they are the sums).
template <int BF16, int NT, int NV, int GATES>
__global__ __launch_bounds__(NT * rows_of<NT>()) void residual_norm_grad_kernel(NormArgs g) {
    constexpr int ROWS = rows_of<NT>();
    constexpr bool AHEAD = NV == 1 || BF16;   // the next row's inputs are on their way (where registers hold them)
    typedef SharedChannels<NT, NV> Vector;
    __shared__ f32x4 channels[3][Vector::SIZE];
    __shared__ float part[2][3][NT / 64];
    __shared__ float across[ROWS > 1 ? 3 * NT * NV * 8 : 1];
    const int tid = threadIdx.x % NT, H = g.H;
    const int64_t step = (int64_t)gridDim.x * ROWS;
    int64_t row = (int64_t)blockIdx.x * ROWS + __builtin_amdgcn_readfirstlane(threadIdx.x / NT);
    const float inv = 1.0f / (float)H;
    int turn = 0;

    const GradInputs<BF16, NT, GATES> of(g, tid);
    typename GradInputs<BF16, NT, GATES>::Piece next[AHEAD ? NV : 1];
    if constexpr (AHEAD) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (row < g.T) next[i] = of.read(row, i);
    }
    const Vector weight(channels[0], g.weight, tid, H), post(channels[1], g.post, tid, H), gate(channels[2], g.gate, tid, H);
    float sum[3][NV][8];
#pragma unroll
    for (int a = 0; a < 3; ++a)
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[a][i][e] = 0.0f;

    for (; row < g.T; row += step) {
        typename GradInputs<BF16, NT, GATES>::Piece in[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) in[i] = of.settled(AHEAD ? next[AHEAD ? i : 0] : of.read(row, i), i);
        if constexpr (AHEAD) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (row + step < g.T) next[i] = of.read(row + step, i);
        }
        auto inputs = [&](int i) {
            if constexpr (BF16) forget(in[i].t), forget(in[i].dz), forget(in[i].y);
            return in[i];
        };
        float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const auto p = inputs(i);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const f32x4 w = weight(i, h);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float t = p.t.at(4 * h + e), y = p.y.at(4 * h + e);
                    s[0] = __builtin_fmaf(t, t, s[0]);
                    s[1] = __builtin_fmaf(p.dz.at(4 * h + e) * w[e], t, s[1]);
                    s[2] = __builtin_fmaf(y, y, s[2]);
                }
            }
            __builtin_amdgcn_sched_barrier(0);   // a piece at a time, which takes fewer registers
        }
        row_sums<NT>(s, part, turn);
        const float r = g.weight ? 1.0f / __builtin_sqrtf(s[0] * inv + g.eps) : 0.0f, mean = s[1] * inv * r;
        const float q = g.post ? 1.0f / __builtin_sqrtf(s[2] * inv + g.eps) : 1.0f;
        // the gradient with respect to t
        auto slope = [&](const auto &p, int e, float w) {
            return __builtin_fmaf(r, __builtin_fmaf(-(p.t.at(e) * r), mean, p.dz.at(e) * w), p.dt.at(e));
        };
        float d[NV][8], dot[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const auto p = inputs(i);
            float out[8], dg[8], dn[8];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const f32x4 w = weight(i, h), b = post(i, h), c = gate(i, h);
#pragma unroll
                for (int f = 0; f < 4; ++f) {
                    const int e = 4 * h + f;
                    const float yh = p.y.at(e) * q, v = slope(p, e, w[f]);
                    sum[0][i][e] = __builtin_fmaf(p.dz.at(e), p.t.at(e) * r, sum[0][i][e]);
                    out[e] = g.scale * v;
                    dg[e] = v * (yh * b[f]);
                    if constexpr (!GATES) sum[2][i][e] += dg[e];
                    dn[e] = v * (GATES ? p.gate.at(e) : c[f]);
                    sum[1][i][e] = __builtin_fmaf(dn[e], yh, sum[1][i][e]);
                    dn[e] *= b[f];
                    dot[0] = __builtin_fmaf(dn[e], yh, dot[0]);
                    d[i][e] = dn[e];
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            store8<BF16>(g.t, row, tid + i * NT, H, out);
            if constexpr (GATES) store8<BF16>(g.dgates, row, tid + i * NT, H, dg);
        }
        if (!g.y) continue;
        float m = 0.0f;
        if (g.post) {
            row_sums<NT>(dot, part, turn);
            m = dot[0] * inv;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const auto p = inputs(i);
            float out[8];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int f = 0; f < 4; ++f) {
                    const int e = 4 * h + f;
                    out[e] = g.post ? q * __builtin_fmaf(-(p.y.at(e) * q), m, d[i][e]) : d[i][e];
                }
            }
            store8<BF16>(g.z, row, tid + i * NT, H, out);
        }
    }

    // one partial row per workgroup; a workgroup's waves add theirs in order
    if constexpr (ROWS > 1) {
#pragma unroll
        for (int w = 0; w < ROWS; ++w) {
            if ((int)threadIdx.x / NT == w) {
#pragma unroll
                for (int a = 0; a < 3; ++a)
#pragma unroll
                    for (int i = 0; i < NV; ++i)
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            float *at = across + ((a * NV + i) * 8 + e) * NT + tid;
                            if (w > 0) sum[a][i][e] += *at;
                            *at = sum[a][i][e];
                        }
            }
            __syncthreads();
        }
        if ((int)threadIdx.x / NT != ROWS - 1) return;
    }
#pragma unroll
    for (int a = 0; a < 3; ++a) {
        if (g.sums[a]) {
#pragma unroll
            for (int i = 0; i < NV; ++i) store8<0>(g.sums[a] + blockIdx.x * g.pitch, 0, tid + i * NT, H, sum[a][i]);
        }
    }
}

// Rows above 8192, whose inputs do not fit the registers beside the sums over the rows: r, mean, q and m of each row
// first (see residual_norm_grad_kernel), a workgroup to a row, then everything else by strips of 2048 channels, the inputs
// read a second time (bf16 2048 x 16384: 65 us for the reads of the first, 4.1 TB/s, 78 us for the second, 5.1). With both in
// one kernel, inputs and vectors read again from the caches for each use, that gradient took 520 us, now 145; with the
// vectors of the first read from the caches for each row 32 us more.
template <int BF16, int GATES>
__global__ __launch_bounds__(512) void norm_grad_rows_kernel(NormArgs g, f32x4 *rows) {
    constexpr int NT = 512, NV = 4;
    typedef SharedChannels<NT, NV> Vector;
    typedef typename GradInputs<BF16, NT, GATES>::Piece Piece;
    __shared__ f32x4 channels[2][Vector::SIZE];
    __shared__ float part[2][3][NT / 64];
    const int tid = threadIdx.x;
    const GradInputs<BF16, NT, GATES> of(g, tid);
    const float inv = 1.0f / (float)g.H;
    int64_t row = blockIdx.x;
    int turn = 0;
    Piece next[BF16 ? NV : 1];   // the next row's (where registers hold them)
    if constexpr (BF16) {
#pragma unroll
        for (int i = 0; i < NV; ++i) next[i] = of.read(row, i);   // (there are no more workgroups than rows)
    }
    const Vector weight(channels[0], g.weight, tid, g.H), post(channels[1], g.post, tid, g.H);   // (post: times the gate)
    if (g.gate) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Raw<0> c = Channels<NT, NV, false>(g.gate, tid, g.H).read(i);
#pragma unroll
            for (int h = 0; h < 2; ++h) post.at[(2 * i + h) * NT + tid] *= __builtin_bit_cast(f32x4, c.v[h]);
        }
    }
    for (; row < g.T; row += gridDim.x) {
        Piece in[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) in[i] = BF16 ? next[BF16 ? i : 0] : of.read(row, i);
#pragma unroll
        for (int i = 0; i < NV; ++i) in[i] = of.settled(in[i], i);
        if constexpr (BF16) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (row + gridDim.x < g.T) next[i] = of.read(row + gridDim.x, i);
        }
        float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const f32x4 w = weight(i, h);
#pragma unroll
                for (int f = 0; f < 4; ++f) {
                    const int e = 4 * h + f;
                    const float t = in[i].t.at(e), y = in[i].y.at(e);
                    s[0] = __builtin_fmaf(t, t, s[0]);
                    s[1] = __builtin_fmaf(in[i].dz.at(e) * w[f], t, s[1]);
                    s[2] = __builtin_fmaf(y, y, s[2]);
                }
            }
            __builtin_amdgcn_sched_barrier(0);   // a piece at a time, which takes fewer registers
        }
        row_sums<NT>(s, part, turn);
        const float r = g.weight ? 1.0f / __builtin_sqrtf(s[0] * inv + g.eps) : 0.0f, mean = s[1] * inv * r;
        const float q = g.post ? 1.0f / __builtin_sqrtf(s[2] * inv + g.eps) : 1.0f;
        float dot[1] = {0.0f};
        if (g.post) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if constexpr (BF16) forget(in[i].t), forget(in[i].dz), forget(in[i].y);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const f32x4 w = weight(i, h), b = post(i, h);
#pragma unroll
                    for (int f = 0; f < 4; ++f) {
                        const int e = 4 * h + f;
                        const float v = __builtin_fmaf(r, __builtin_fmaf(-(in[i].t.at(e) * r), mean, in[i].dz.at(e) * w[f]), in[i].dt.at(e));
                        dot[0] = __builtin_fmaf(GATES ? v * in[i].gate.at(e) * b[f] : v * b[f], in[i].y.at(e) * q, dot[0]);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            row_sums<NT>(dot, part, turn);
        }
        if (tid == 0) rows[row] = f32x4{r, mean, q, dot[0] * inv};
    }
}

template <int BF16, int GATES>
__global__ __launch_bounds__(256) void norm_grad_strips_kernel(NormArgs g, const f32x4 *rows) {
    constexpr int NT = 256;
    const int tid = blockIdx.x * NT + threadIdx.x;   // this thread's piece of every row
    const GradInputs<BF16, NT, GATES> of(g, tid);
    typedef Channels<NT, 1, true> Vector;
    const Vector weight(g.weight, tid, g.H), post(g.post, tid, g.H), gate(g.gate, tid, g.H);
    const Raw<0> w = weight(0), b = post(0), c = gate(0);
    float sum[3][8];
#pragma unroll
    for (int a = 0; a < 3; ++a)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[a][e] = 0.0f;
    int64_t row = blockIdx.y;
    typename GradInputs<BF16, NT, GATES>::Piece next = of.read(row, 0);   // (there are no more workgroups than rows)
    for (; row < g.T; row += gridDim.y) {
        const auto p = of.settled(next, 0);
        if (row + gridDim.y < g.T) next = of.read(row + gridDim.y, 0);
        const f32x4 of_row = rows[row];
        const float r = of_row[0], mean = of_row[1], q = of_row[2], m = of_row[3];
        float out[8], dg[8], dy[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float yh = p.y.at(e) * q;
            const float v = __builtin_fmaf(r, __builtin_fmaf(-(p.t.at(e) * r), mean, p.dz.at(e) * w.at(e)), p.dt.at(e));
            sum[0][e] = __builtin_fmaf(p.dz.at(e), p.t.at(e) * r, sum[0][e]);
            out[e] = g.scale * v;
            dg[e] = v * (yh * b.at(e));
            if constexpr (!GATES) sum[2][e] += dg[e];
            const float dn = v * (GATES ? p.gate.at(e) : c.at(e));
            sum[1][e] = __builtin_fmaf(dn, yh, sum[1][e]);
            dy[e] = g.post ? q * __builtin_fmaf(-yh, m, dn * b.at(e)) : dn;
        }
        store8<BF16>(g.t, row, tid, g.H, out);
        if constexpr (GATES) store8<BF16>(g.dgates, row, tid, g.H, dg);
        if (g.y) store8<BF16>(g.z, row, tid, g.H, dy);
    }
#pragma unroll
    for (int a = 0; a < 3; ++a)
        if (g.sums[a]) store8<0>(g.sums[a] + blockIdx.y * g.pitch, 0, tid, g.H, sum[a]);
}

// The partial rows added up: 64 channels a workgroup, 16 threads to a channel (256 partials of 3 x 7168 5 us, from the
// caches)
__global__ __launch_bounds__(1024) void norm_sums_kernel(const float *partials, int64_t n, int H, float *o0, float *o1,
                                                         float *o2) {
    __shared__ float part[16][64];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, a = blockIdx.y;
    float *const out = a == 0 ? o0 : a == 1 ? o1 : o2;
    const int col = blockIdx.x * 64 + lane;
    float s = 0.0f;
    if (out && col < H) {
        const float *p = partials + (int64_t)a * H + col;
#pragma unroll 8
        for (int64_t i = w; i < n; i += 16) s += p[i * 3 * H];
    }
    part[w][lane] = s;
    __syncthreads();
    if (w == 0 && out && col < H) {
#pragma unroll
        for (int i = 1; i < 16; ++i) s += part[i][lane];
        out[col] = s;
    }
}

// calls f.run<NT, NV>() for rows of H elements, those above 4096 by MID threads, or f.run_long() above 8192
template <int MID, class F>
void for_length(int H, const F &f) {
    if (H <= 512) f.template run<64, 1>();
    else if (H <= 1024) f.template run<128, 1>();
    else if (H <= 2048) f.template run<256, 1>();
    else if (H <= 4096) f.template run<512, 1>();
    else if (H <= 8192) f.template run<MID, 8192 / 8 / MID>();
    else f.run_long();
}

constexpr int64_t kCUs = 256;

template <int BF16>
struct Forward {
    const NormArgs &a;
    hipStream_t stream;
    template <int NT, int NV>
    void run() const {
        constexpr int THREADS = NT * rows_of<NT>();
        const int64_t need = (a.T + rows_of<NT>() - 1) / rows_of<NT>(), most = kCUs * (1024 / THREADS);
        const dim3 grid((unsigned)(need < most ? need : most));
        if (a.gates) residual_norm_kernel<BF16, NT, NV, 1><<<grid, dim3(THREADS), 0, stream>>>(a);
        else residual_norm_kernel<BF16, NT, NV, 0><<<grid, dim3(THREADS), 0, stream>>>(a);
    }
    void run_long() const { run<1024, 2>(); }
};

template <int BF16>
struct Backward {
    const NormArgs &a;
    int64_t workgroups;
    f32x4 *rows;
    hipStream_t stream;
    template <int NT, int NV>
    void run() const {
        const dim3 grid((unsigned)workgroups), block(NT * rows_of<NT>());
        if (a.gates) residual_norm_grad_kernel<BF16, NT, NV, 1><<<grid, block, 0, stream>>>(a);
        else residual_norm_grad_kernel<BF16, NT, NV, 0><<<grid, block, 0, stream>>>(a);
    }
    template <int GATES>
    void strips() const {
        norm_grad_rows_kernel<BF16, GATES><<<dim3((unsigned)(a.T < kCUs ? a.T : kCUs)), dim3(512), 0, stream>>>(a, rows);
        norm_grad_strips_kernel<BF16, GATES><<<dim3((a.H + 2047) / 2048, (unsigned)workgroups), dim3(256), 0, stream>>>(a, rows);
    }
    void run_long() const {
        if (a.gates) strips<1>();
        else strips<0>();
    }
};

// Workgroups of the gradient, each of which leaves a partial row: as many as run at once, where that is worth
// their partials. us with 256 / 512 / 1024 of them, bf16: 4096 x 7168 94 / 103 / 129, 4096 x 2048 34 / 28 / 32,
// 4096 x 1024 33 / 24 / 21, 16384 x 512 30 / 26 / 29, 1024 x 1091 15 / 16 / 22. Of strips of long rows three workgroups a
// CU run at once; us with 96 / 128 / 256 to a strip: bf16 2048 x 16384 (8 strips) 145 / 157 / 154, fp32 2048 x 12288 (6)
// 233 / 215 / 216.
int64_t grad_workgroups(int64_t T, int64_t H) {
    const int64_t need = H <= 512 ? (T + 3) / 4 : T;
    const int64_t most = H > 8192 ? 3 * kCUs / ((H + 2047) / 2048) : H > 2048 ? kCUs
                         : H > 512 && H <= 1024 && T >= 4096 ? 4 * kCUs : T >= 1536 ? 2 * kCUs : kCUs;
    return need < most ? need : most;
}

}  // namespace

hipError_t launch_residual_norm(const void *x, const void *y, bool bf16, const float *weight, const float *post,
                                const float *gate, const void *gates, float scale, float eps, void *t, void *z,
                                int64_t T, int64_t H, hipStream_t stream) {
    NormArgs a{};
    a.x = x, a.y = y, a.weight = weight, a.post = post, a.gate = gate, a.gates = gates, a.scale = scale, a.eps = eps;
    a.t = t, a.z = z, a.T = T, a.H = (int)H;
    if (bf16) for_length<1024>((int)H, Forward<1>{a, stream});
    else for_length<1024>((int)H, Forward<0>{a, stream});
    return hipGetLastError();
}

size_t residual_norm_grad_workspace_bytes(int64_t T, int64_t H) {
    const int64_t n = grad_workgroups(T, H);
    return (size_t)((n > 1 ? n * 3 * H * 4 : 0) + (H > 8192 ? 16 * T : 0));
}

hipError_t launch_residual_norm_backward(const void *dt, const void *dz, const void *t, const void *y, bool bf16,
                                         const float *weight, const float *post, const float *gate, const void *gates,
                                         float scale, float eps, void *dx, void *dy, float *dweight, float *dpost,
                                         float *dgate, void *dgates, int64_t T, int64_t H, void *workspace,
                                         hipStream_t stream) {
    NormArgs a{};
    a.x = t, a.y = y, a.dt = dt, a.dz = dz, a.weight = weight, a.post = post, a.gate = gate, a.gates = gates;
    a.scale = scale, a.eps = eps, a.t = dx, a.z = dy, a.dgates = dgates, a.T = T, a.H = (int)H;
    const int64_t n = grad_workgroups(T, H);
    f32x4 *const rows = static_cast<f32x4 *>(workspace);   // (of long rows only)
    float *const out[3] = {dweight, dpost, dgate}, *const partials = reinterpret_cast<float *>(rows + (H > 8192 ? T : 0));
    for (int i = 0; i < 3; ++i) a.sums[i] = out[i] ? (n > 1 ? partials + i * H : out[i]) : nullptr;
    a.pitch = 3 * H;
    if (n > 0) {
        if (bf16) for_length<512>((int)H, Backward<1>{a, n, rows, stream});
        else for_length<512>((int)H, Backward<0>{a, n, rows, stream});
        if (hipError_t e = hipGetLastError()) return e;
    }
    if (n == 1 || !(dweight || dpost || dgate)) return hipSuccess;
    // (with no rows the sums are zero)
    norm_sums_kernel<<<dim3((unsigned)((H + 63) / 64), 3), dim3(1024), 0, stream>>>(partials, n, (int)H, dweight, dpost,
                                                                                   dgate);
    return hipGetLastError();
}

}  // namespace fp8q
