// gated.hip -- the gated projection of a feed-forward block: both projections, the activation and the
// product in one kernel, and its gradient, for gfx950.
//
//     g = x Wg^T, u = x Wu^T  (W = [Wg; Wu]),  h = act(g) * u
//     dg = dh * u * act'(g),  du = dh * act(g),  dx = [dg du] W,  dW = [dg du]^T x
//
// act is SiLU, a / (1 + e^-a), or GELU, a * Phi(a) with Phi by erfc (which keeps its relative precision
// where Phi is small). Products are bf16 with fp32 sums (mm.h); activation and product are fp32 on the
// sums, rounded once. The gradient's products take dg and du rounded to bf16, the matrix unit's type, or where the
// caller asks for more (`wide`) as two bf16 numbers, the rounded one and what it lost (16 bits in all), each with
// products of its own. Error of a bf16 output against 64 bits 2.3e-3 rms rounded, 1.7e-3 (the output's own rounding) wide;
// 4096 x 7168 -> 2048 397 / 1060 us, 1021 x 1536 -> 4096 102 / 213, 16 x 128 -> 128 7.5 / 10.
//
// The projections' columns are dealt so that a lane holds g and u of the same element: nothing of them
// goes through memory unless the caller keeps them. The gradient forms dg and du from kept projections (a
// pass over memory) or by the same product again with another epilogue, then takes two products whose
// operands are transposed by their LDS reads.
//
// Bound by the matrix unit, and there by the power it may take: 8192 x 7168 -> 2048 327 us on the device, 1.47 PFLOP/s,
// the unit busy 0.75; the gradient's products of 4096 rows 378 us, 1.27 PFLOP/s, busy 0.58 (twice the LDS reads, of 8
// bytes). Few rows are bound by the read of W: 1 x 7168 -> 2048 9 us, 6.5 TB/s.
#include <cmath>

#include <fp8q.h>

#include "mm.h"

namespace fp8q {
namespace {

struct GatedArgs {
    MmArgs mm;            // N = F
    void *h;              // [M, F]
    uint16_t *gu;         // [M, 2 F] or null; the gradient: dg and du
    const uint16_t *dh;   // the gradient: [M, F]
    uint16_t *rest;       // the gradient: what dg and du lose in gu, [M, 2 F], or null
    int gelu;
};

// The activation and its slope, with the hardware's exponential and reciprocal (each within one unit in the last
// place) and the roundings of their arguments put right, which a large argument would otherwise pass on
// multiplied: some 20 to 35 operations. (expf, erfcf and the division took 100 and more, and a tile has 64 of
// these a lane: the projections of 1021 x 1536 -> 4096 with GELU's gradient 36 us, now 33.5.)
constexpr float kLog2e = 1.44269502f, kLog2eRest = 1.92596299e-8f, kLn2 = 0.693147182f;
__device__ __forceinline__ float reciprocal(float d) {
    const float r = __builtin_amdgcn_rcpf(d);
    return __builtin_fmaf(__builtin_fmaf(-d, r, 1.0f), r, r);
}
// e^-(v + rest) times 2^shift, v up to 113, rest a rounding of v; shift 0, or 64 where v is above 64: it then makes
// the exponent smaller, which is exact
__device__ __forceinline__ float exp_minus(float v, float rest, float shift) {
    const float t = -v * kLog2e;
    const float off = __builtin_fmaf(-v, kLog2e, -t) - __builtin_fmaf(v, kLog2eRest, rest * kLog2e);
    const float e = __builtin_amdgcn_exp2f(t + shift);
    return __builtin_fmaf(e * kLn2, off, e);
}
// Far below zero the exponential leaves the normal numbers before its product with a does. There it is carried with a
// factor of 2^64, which comes off last: by SiLU in a branch of its own below -87 (done for every a, 4096 x 512 -> 4096
// took 50.4 us instead of 45.2), by GELU for the slope alone, whose value there is no normal number.
constexpr float kFarSilu = -87.0f, kFar = 64.0f, kBack = 0x1p-64f;

// four of them; slope is left as it is without SLOPE
template <bool SLOPE>
__device__ __forceinline__ void silu4(const f32x4 &a, f32x4 &value, f32x4 &slope) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        float p = reciprocal(1.0f + exp_minus(__builtin_amdgcn_fmed3f(a[r], kFarSilu, -kFarSilu), 0.0f, 0.0f));
        p = a[r] == a[r] ? p : a[r];
        value[r] = a[r] * p;
        if constexpr (SLOPE) slope[r] = p * __builtin_fmaf(a[r], 1.0f - p, 1.0f);
    }
    if ((a[0] < kFarSilu) | (a[1] < kFarSilu) | (a[2] < kFarSilu) | (a[3] < kFarSilu)) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            // (e^a / (1 + e^a) is e^a here; below -110 nothing is left of it)
            const float e = a[r] < -110.0f ? 0.0f : exp_minus(-a[r], 0.0f, kFar);
            value[r] = a[r] < kFarSilu ? a[r] * e * kBack : value[r];
            if constexpr (SLOPE) slope[r] = a[r] < kFarSilu ? e * (1.0f + a[r]) * kBack : slope[r];
        }
    }
}
// Phi(a) = erfc(-a / sqrt 2) / 2; for negative a, e^(-a^2 / 2) / 2 times erfc's other factor, a polynomial in
// 1 / (1 + |a| / sqrt 8) (its coefficients, as they stand here, within 5.1e-8 relative up to 13.2, where a Phi(a) leaves
// the normal numbers); from 14.5 on it is 0
template <bool SLOPE>
__device__ __forceinline__ void gelu4(const f32x4 &a, f32x4 &value, f32x4 &slope) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const float c = __builtin_amdgcn_fmed3f(a[r], -15.0f, 15.0f), half = 0.5f * c, v = c * half;
        const bool far = SLOPE && v > kFar;
        const float e = exp_minus(v, __builtin_fmaf(c, half, -v), far ? kFar : 0.0f), back = far ? kBack : 1.0f;
        const float w = reciprocal(__builtin_fmaf(__builtin_fabsf(c), 0.353553391f, 1.0f));
        float g = -0.0540772378f;
        g = __builtin_fmaf(g, w, 0.258805364f);
        g = __builtin_fmaf(g, w, -0.429980040f);
        g = __builtin_fmaf(g, w, 0.206562728f);
        g = __builtin_fmaf(g, w, 0.0286144651f);
        g = __builtin_fmaf(g, w, 0.175417840f);
        g = __builtin_fmaf(g, w, 0.251677930f);
        g = __builtin_fmaf(g, w, 0.280724078f);
        g = __builtin_fmaf(g, w, 0.282262772f);
        g = __builtin_fmaf(g, w, -7.95229838e-6f);
        const float q = 0.5f * e * g * back;
        float p = c > 0.0f ? 1.0f - q : q;
        p = a[r] == a[r] ? p : a[r];
        value[r] = a[r] * p;
        if constexpr (SLOPE) slope[r] = __builtin_fmaf(c * (e * 0.398942280f), back, p);
    }
}
template <bool SLOPE>
__device__ __forceinline__ void activate4(const f32x4 &a, int gelu, f32x4 &value, f32x4 &slope) {
    if (gelu) gelu4<SLOPE>(a, value, slope);
    else silu4<SLOPE>(a, value, slope);
}

// What v loses when it is rounded to bf16 (nothing where that is not finite: infinities stay the first number's)
__device__ __forceinline__ float rest_of(float v) {
    const float r = bf16lo_to_f32(pack_bf16x2(v, 0.0f));
    return __builtin_fabsf(r) < __builtin_inff() ? v - r : 0.0f;
}
__device__ __forceinline__ f32x4 rest_of(const f32x4 &v) { return f32x4{rest_of(v[0]), rest_of(v[1]), rest_of(v[2]), rest_of(v[3])}; }

// MODE 0, 1: h in fp32, bf16; 2: dg and du
template <class T, int MODE>
__device__ __forceinline__ void gated_tile(const GatedArgs &g, int64_t m0, int64_t n0, uint8_t *smem) {
    constexpr int HALF = T::SUB_N / 2;
    f32x4 acc[T::SUB_M][T::SUB_N];
    multiply<T, 0, 0, 1, MODE>(g.mm, m0, n0, smem, acc, []() {});
    const int64_t M = g.mm.M, F = g.mm.N;
    auto gate = [&](int i, int j) { return acc[i][j]; };
    auto up = [&](int i, int j) { return acc[i][j + HALF]; };
    if constexpr (MODE == 2) {
        const int lane = threadIdx.x & 63, wm = wave_m<T>(), wn = wave_n<T>();
#pragma unroll
        for (int i = 0; i < T::SUB_M; ++i) {
            const int64_t m = m0 + T::row(wm, i) + (lane & 15);
#pragma unroll
            for (int j = 0; j < HALF; ++j) {
                const int64_t n = n0 + 16 * (wn * HALF + j) + 4 * (lane >> 4);
                f32x4 dh = {0.f, 0.f, 0.f, 0.f};
                if (m < M && n < F) dh = load4<1>(g.dh, m * F + n, F - n);
                f32x4 value, slope;
                activate4<true>(acc[i][j], g.gelu, value, slope);
                acc[i][j] = dh * acc[i][j + HALF] * slope;
                acc[i][j + HALF] = dh * value;
            }
            __builtin_amdgcn_sched_barrier(0);   // (16 rows at a time, as the registers allow)
        }
    } else {
        store_tile<T, MODE, HALF>(g.h, F, m0, M, n0, F, smem, [&](int i, int j) {
            f32x4 value, none;
            activate4<false>(acc[i][j], g.gelu, value, none);
            return value * acc[i][j + HALF];
        });
    }
    if (g.gu) {
        store_tile<T, 1, HALF>(g.gu, 2 * F, m0, M, n0, F, smem, gate);
        store_tile<T, 1, HALF>(g.gu + F, 2 * F, m0, M, n0, F, smem, up);
    }
    if constexpr (MODE == 2) {
        if (g.rest) {
            store_tile<T, 1, HALF>(g.rest, 2 * F, m0, M, n0, F, smem, [&](int i, int j) { return rest_of(acc[i][j]); });
            store_tile<T, 1, HALF>(g.rest + F, 2 * F, m0, M, n0, F, smem, [&](int i, int j) { return rest_of(acc[i][j + HALF]); });
        }
    }
}

template <int BM, int BN, int NW, int NSTAGE, int MODE>
__global__ __launch_bounds__(NW * 64) __attribute__((amdgpu_waves_per_eu(NW == 8 ? 2 : 1, 2))) void gated_kernel(GatedArgs g) {
    using T = Tile<BM, BN, NW, 2, NSTAGE>;
    __shared__ __attribute__((aligned(16))) uint8_t smem[T::STAGE * NSTAGE];
    int64_t m0, n0;
    find_tile<T, BN / 2>(g.mm, m0, n0);
    gated_tile<T, MODE>(g, m0, n0, smem);
}

constexpr int kShareBytes = HalfTile::STAGE * HalfTile::NSTAGE;
static_assert(kShareBytes >= WholeTile::STAGE * WholeTile::NSTAGE, "LDS of both");
template <int MODE>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void gated_large_kernel(GatedArgs g) {
    __shared__ __attribute__((aligned(16))) uint8_t smem[kShareBytes];
    bool second;
    int tile, half;
    if (!find_share(g.mm.tiles_m * g.mm.tiles_n, 0, second, tile, half)) return;
    int64_t m0, n0;
    place_tile(g.mm, tile, 256, 128, m0, n0);
    if (half < 0) {
        gated_tile<WholeTile, MODE>(g, m0, n0, smem);
    } else {
        m0 += 128 * half;
        if (m0 < g.mm.M) gated_tile<HalfTile, MODE>(g, m0, n0, smem);
    }
}

// At most 16 RX rows
template <int RX, int NB, int MODE>
__global__ __launch_bounds__(256) void gated_few_kernel(GatedArgs g) {
    __shared__ __attribute__((aligned(16))) uint8_t smem[Few<RX, NB>::BYTES];
    constexpr int COLS = NB / 2;
    const int64_t n0 = (int64_t)blockIdx.x * COLS, F = g.mm.N;
    const float *const sums = few<RX, NB, 1, MODE>(g.mm, n0, smem, []() {});
    const int p = threadIdx.x, row = p / (COLS / 4), at = 4 * (p % (COLS / 4));
    static_assert(16 * RX * COLS / 4 <= 256, "four columns a thread");
    const int64_t m = row, n = n0 + at;
    if (row >= 16 * RX || m >= g.mm.M || n >= F) return;
    const f32x4 gate = *reinterpret_cast<const f32x4 *>(sums + row * NB + at);
    const f32x4 up = *reinterpret_cast<const f32x4 *>(sums + row * NB + COLS + at);
    f32x4 value, slope;
    activate4<MODE == 2>(gate, g.gelu, value, slope);
    if constexpr (MODE == 2) {
        const f32x4 dh = load4<1>(g.dh, m * F + n, F - n), a = dh * up * slope, b = dh * value;
        store4<1>(g.gu, m * 2 * F + n, a, F - n);
        store4<1>(g.gu, (m * 2 + 1) * F + n, b, F - n);
        if (g.rest) {
            store4<1>(g.rest, m * 2 * F + n, rest_of(a), F - n);
            store4<1>(g.rest, (m * 2 + 1) * F + n, rest_of(b), F - n);
        }
    } else {
        store4<MODE>(g.h, m * F + n, value * up, F - n);
        if (g.gu) {
            store4<1>(g.gu, m * 2 * F + n, gate, F - n);
            store4<1>(g.gu, (m * 2 + 1) * F + n, up, F - n);
        }
    }
}

// dg and du from kept projections, 8 elements a thread (F is a multiple of 8): bound by memory (4096 x 2048 15.5 us,
// 5.4 TB/s, some of it from the caches)
template <bool WIDE>
__global__ __launch_bounds__(256) void gated_slope_kernel(const uint16_t *dh, const uint16_t *gu, uint16_t *d, uint16_t *rest,
                                                          int64_t n, int64_t F, int gelu) {
    const int64_t step = (int64_t)gridDim.x * 256, per = F / 8;
    for (int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x; p < n; p += step) {
        const int64_t m = p / per, at = m * 2 * F + 8 * (p - m * per);
        const u32x4 vh = *reinterpret_cast<const u32x4 *>(dh + 8 * p), vg = *reinterpret_cast<const u32x4 *>(gu + at),
                    vu = *reinterpret_cast<const u32x4 *>(gu + at + F);
        u32x4 a, b, ra, rb;
        auto four = [](const u32x4 &v, int i) {   // elements 2 i .. 2 i + 3
            return f32x4{bf16lo_to_f32(v[i]), bf16hi_to_f32(v[i]), bf16lo_to_f32(v[i + 1]), bf16hi_to_f32(v[i + 1])};
        };
        auto put = [](u32x4 &to, int i, const f32x4 &v) { to[i] = pack_bf16x2(v[0], v[1]), to[i + 1] = pack_bf16x2(v[2], v[3]); };
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            f32x4 value, slope;
            activate4<true>(four(vg, i), gelu, value, slope);
            const f32x4 h = four(vh, i), dg = h * four(vu, i) * slope, du = h * value;
            put(a, i, dg), put(b, i, du);
            if constexpr (WIDE) put(ra, i, rest_of(dg)), put(rb, i, rest_of(du));
        }
        *reinterpret_cast<u32x4 *>(d + at) = a;
        *reinterpret_cast<u32x4 *>(d + at + F) = b;
        if constexpr (WIDE) {
            *reinterpret_cast<u32x4 *>(rest + at) = ra;
            *reinterpret_cast<u32x4 *>(rest + at + F) = rb;
        }
    }
}

// The gradient's products, dW = d^T x and dx = d W, in one launch: W's operand is K-strided in both, X's in dW's (XT).
// K in `splits` parts, each a set of tiles of its own, whose sums go to y + part * M * N and are added by a
// second kernel. With two pieces the parts of d's rests, `rest` elements behind d, follow those of d.
struct ProductArgs {
    MmArgs mm;
    void *y;
    int bf16, splits;   // splits 0: not wanted
    int pieces;
    int64_t rest;
};
__host__ __device__ __forceinline__ int tiles_of(const ProductArgs &g) { return g.mm.tiles_m * g.mm.tiles_n * g.splits * g.pieces; }

template <class T, int XT, int TAG>
__device__ __forceinline__ void grad_tile(const ProductArgs &g, int64_t m0, int64_t n0, uint8_t *smem) {
    f32x4 acc[T::SUB_M][T::SUB_N];
    multiply<T, XT, 1, 0, TAG>(g.mm, m0, n0, smem, acc, []() {});
    auto value = [&](int i, int j) { return acc[i][j]; };
    if (g.bf16) store_tile<T, 1, T::SUB_N>(g.y, g.mm.N, m0, g.mm.M, n0, g.mm.N, smem, value);
    else store_tile<T, 0, T::SUB_N>(g.y, g.mm.N, m0, g.mm.M, n0, g.mm.N, smem, value);
}

template <class T, int XT, int TAG>
__device__ __forceinline__ void grad_part(ProductArgs g, int tile, uint8_t *smem) {
    const int n = g.mm.tiles_m * g.mm.tiles_n, part = tile / n;
    int64_t m0, n0;
    place_tile(g.mm, tile - part * n, T::BM, T::BN, m0, n0);
    if (g.splits * g.pieces > 1) {
        const int64_t steps = (g.mm.K + KSTEP - 1) / KSTEP;
        const int piece = part / g.splits, of = part - piece * g.splits;
        const int64_t k0 = of * steps / g.splits * KSTEP, k1 = (of + 1) * steps / g.splits * KSTEP;
        g.mm.x += (XT ? k0 * g.mm.ldx : k0) + piece * g.rest;
        g.mm.w += k0 * g.mm.ldw;
        g.mm.K = (k1 < g.mm.K ? k1 : g.mm.K) - k0;
        g.y = static_cast<float *>(g.y) + part * g.mm.M * g.mm.N;
        g.bf16 = 0;
    }
    grad_tile<T, XT, TAG>(g, m0, n0, smem);
}

// Each XCD takes a contiguous run of dW's tiles, then one of dx's
template <int BM, int BN, int NW, int NSTAGE>
__global__ __launch_bounds__(NW * 64) __attribute__((amdgpu_waves_per_eu(NW == 8 ? 2 : 1, 2))) void gated_grads_kernel(ProductArgs dw, ProductArgs dx) {
    using T = Tile<BM, BN, NW, 2, NSTAGE>;
    __shared__ __attribute__((aligned(16))) uint8_t smem[T::STAGE * NSTAGE];
    const int xcd = blockIdx.x & 7, slot = blockIdx.x >> 3;
    const int w0 = run_of(tiles_of(dw), xcd), w = run_of(tiles_of(dw), xcd + 1) - w0;
    const int x0 = run_of(tiles_of(dx), xcd), x = run_of(tiles_of(dx), xcd + 1) - x0;
    if (slot < w) grad_part<T, 1, 4>(dw, w0 + slot, smem);
    else if (slot < w + x) grad_part<T, 0, 4>(dx, x0 + slot - w, smem);
}

// The largest tiles, K whole
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void gated_grads_large_kernel(ProductArgs dw, ProductArgs dx) {
    __shared__ __attribute__((aligned(16))) uint8_t smem[kShareBytes];
    bool second;
    int tile, half;
    if (!find_share(tiles_of(dw), tiles_of(dx), second, tile, half)) return;
    int64_t m0, n0;
    if (second) {
        place_tile(dx.mm, tile, 256, 256, m0, n0);
        if (half < 0) {
            grad_tile<WholeTile, 0, 5>(dx, m0, n0, smem);
        } else {
            m0 += 128 * half;
            if (m0 < dx.mm.M) grad_tile<HalfTile, 0, 5>(dx, m0, n0, smem);
        }
    } else {
        place_tile(dw.mm, tile, 256, 256, m0, n0);
        if (half < 0) {
            grad_tile<WholeTile, 1, 5>(dw, m0, n0, smem);
        } else {
            m0 += 128 * half;
            if (m0 < dw.mm.M) grad_tile<HalfTile, 1, 5>(dw, m0, n0, smem);
        }
    }
}

// The parts' sums added in order, 8 elements a thread (their number is a multiple of 8), of either product that has
// parts; y: where they go. Of two pieces, the second's sums (half the parts) are added where the first's are finite: an
// infinite weight times a rest of 0, or of the other sign, would make NaN of an infinity.
struct SumArgs {
    const float *parts[2];
    void *y[2];
    int64_t n[2];   // 0: no parts
    int bf16[2], splits[2];
    int pieces;
};
__global__ __launch_bounds__(256) void gated_sum_kernel(SumArgs g) {
    const int64_t step = (int64_t)gridDim.x * 256 * 8;
    for (int64_t p = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; p < g.n[0] + g.n[1]; p += step) {
        const int which = p >= g.n[0];
        const int64_t at = which ? p - g.n[0] : p, n = which ? g.n[1] : g.n[0];
        const float *from = (which ? g.parts[1] : g.parts[0]) + at;
        const int splits = which ? g.splits[1] : g.splits[0];
        void *const y = which ? g.y[1] : g.y[0];
        f32x4 a = {0.f, 0.f, 0.f, 0.f}, b = a;
        for (int s = 0; s < splits; ++s) {
            a += *reinterpret_cast<const f32x4 *>(from + s * n);
            b += *reinterpret_cast<const f32x4 *>(from + s * n + 4);
        }
        if (g.pieces > 1) {
            f32x4 c = {0.f, 0.f, 0.f, 0.f}, d = c;
            for (int s = splits; s < 2 * splits; ++s) {
                c += *reinterpret_cast<const f32x4 *>(from + s * n);
                d += *reinterpret_cast<const f32x4 *>(from + s * n + 4);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                a[r] = __builtin_fabsf(a[r]) < __builtin_inff() ? a[r] + c[r] : a[r];
                b[r] = __builtin_fabsf(b[r]) < __builtin_inff() ? b[r] + d[r] : b[r];
            }
        }
        if (which ? g.bf16[1] : g.bf16[0]) {
            *reinterpret_cast<u32x4_any *>(static_cast<uint16_t *>(y) + at) = u32x4{
                pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(b[0], b[1]), pack_bf16x2(b[2], b[3])};
        } else {
            *reinterpret_cast<u32x4_any *>(static_cast<float *>(y) + at) = __builtin_bit_cast(u32x4, a);
            *reinterpret_cast<u32x4_any *>(static_cast<float *>(y) + at + 4) = __builtin_bit_cast(u32x4, b);
        }
    }
}

template <int BM, int BN, int NW, int NSTAGE>
hipError_t launch_gated_tile(GatedArgs a, int mode, hipStream_t stream) {
    if (!lay_out(a.mm, BM, BN / 2, NW * 64)) return hipErrorInvalidValue;
    const dim3 grid((unsigned)(a.mm.tiles_m * a.mm.tiles_n)), block(NW * 64);
    if (mode == 0) gated_kernel<BM, BN, NW, NSTAGE, 0><<<grid, block, 0, stream>>>(a);
    else if (mode == 1) gated_kernel<BM, BN, NW, NSTAGE, 1><<<grid, block, 0, stream>>>(a);
    else gated_kernel<BM, BN, NW, NSTAGE, 2><<<grid, block, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_gated_large(GatedArgs a, int mode, hipStream_t stream) {
    if (!lay_out(a.mm, 256, 128, 512, kShareMore)) return hipErrorInvalidValue;
    const dim3 grid(share_grid(a.mm.tiles_m * a.mm.tiles_n, 0)), block(512);
    if (mode == 0) gated_large_kernel<0><<<grid, block, 0, stream>>>(a);
    else if (mode == 1) gated_large_kernel<1><<<grid, block, 0, stream>>>(a);
    else gated_large_kernel<2><<<grid, block, 0, stream>>>(a);
    return hipGetLastError();
}

template <int RX, int NB>
hipError_t launch_gated_few(const GatedArgs &a, int mode, hipStream_t stream) {
    const dim3 grid((unsigned)((a.mm.N + NB / 2 - 1) / (NB / 2))), block(256);
    if (mode == 0) gated_few_kernel<RX, NB, 0><<<grid, block, 0, stream>>>(a);
    else if (mode == 1) gated_few_kernel<RX, NB, 1><<<grid, block, 0, stream>>>(a);
    else gated_few_kernel<RX, NB, 2><<<grid, block, 0, stream>>>(a);
    return hipGetLastError();
}

// The projections' tiles: few rows (of X) or a tile, and their number
struct GatedTile {
    int bm, bn, threads;
    double first, more, end;
};
constexpr GatedTile kGatedTiles[5] = {{32, 64, 256, 0.155, 0.125, 1.1}, {64, 64, 256, 0.21, 0.18, 1.4}, {128, 128, 256, 0.45, 0.53, 5.0},
                                      {128, 256, 512, 0.75, 0.83, 5.7}, {256, 256, 512, 1.3, 1.5, 8.0}};
enum { kFew16 = 5, kFew32, kFew32Twice };   // 16 rows against 16 or 32 rows of W, 32 rows against 32
int gated_choice(int64_t M, int64_t F, int64_t K) {
    // few rows against the tiles, us: 24 x 3584 x 7168 20.7 / 27.6, 24 x 768 x 7168 13.9 / 17.2, 48 x 3584 x 7168 (four
    // blocks of rows) 30.0 / 26.1
    if (M <= 16) return F <= 2048 ? kFew16 : kFew32;
    if (M <= 32) return kFew32Twice;
    int best = 4;
    double least = HUGE_VAL;
    for (int t = 0; t < 5; ++t) {
        const GatedTile &tile = kGatedTiles[t];
        const double us = tile_time(M, 2 * F, (K + KSTEP - 1) / KSTEP, tile.bm, tile.bn, tile.first, tile.more, tile.end, t == 4);
        if (us < least) least = us, best = t;
    }
    return best;
}

hipError_t launch_gated(const GatedArgs &a, int mode, hipStream_t stream) {
    switch (gated_choice(a.mm.M, a.mm.N, a.mm.K)) {
    case kFew16: return launch_gated_few<1, 16>(a, mode, stream);
    case kFew32: return launch_gated_few<1, 32>(a, mode, stream);
    case kFew32Twice: return launch_gated_few<2, 32>(a, mode, stream);
    case 0: return launch_gated_tile<32, 64, 4, 6>(a, mode, stream);
    case 1: return launch_gated_tile<64, 64, 4, 5>(a, mode, stream);
    case 2: return launch_gated_tile<128, 128, 4, 4>(a, mode, stream);
    case 3: return launch_gated_tile<128, 256, 8, 3>(a, mode, stream);
    default: return launch_gated_large(a, mode, stream);
    }
}

// The gradient's tiles and the parts of its products' K, by their time (us): up to 256 tiles run at once, one a CU, each
// K's steps and an epilogue; more of them take turns. Parts cost the writing and reading of their sums (mostly from the
// caches) and a launch. The constants are fitted to times at 4096, 2048, 1021, 256 and 64 tokens of 7168 and 1536 channels
// and 512 to 4096 hidden ones, with 1 to 8 parts; K-strided X (dW) takes a tenth longer. Both products in one launch, by
// one kind of tile, or each by its own: 1021 tokens, 1536 -> 4096 78 / 70 us, 1000 x 1096 -> 1000 26 / 33.
constexpr int kMaxParts = 8, kLargest = 3;
struct GradTile {
    int bm, bn, threads;
    double first, more, end;
};
constexpr GradTile kGradTiles[kLargest + 1] = {{64, 64, 256, 0.21, 0.19, 0.8}, {128, 128, 256, 0.43, 0.46, 3.5},
                                               {128, 256, 512, 0.78, 0.82, 5.7}, {256, 256, 512, 1.25, 1.35, 8.0}};
using Plan = GatedGradPlan;
// (only plans whose workgroups a grid holds; with none us stays infinite)
Plan plan_of(int64_t M, int64_t F, int64_t K, int pieces, bool has_w, bool has_x) {
    Plan best = {kLargest, has_w, has_x, HUGE_VAL};
    // What does not depend on the other product's parts: K's steps of a part, and what its sums cost
    struct Parts {
        int least, most;
        double steps[kMaxParts + 1], sums[kMaxParts + 1];
        Parts(bool has, int64_t k_steps, double longer, int64_t outputs, int pieces) : least(has), most(0) {
            steps[0] = sums[0] = 0.0;
            if (!has) return;
            most = k_steps < 8 ? 1 : k_steps / 4 < kMaxParts ? (int)(k_steps / 4) : kMaxParts;
            for (int s = 1; s <= most; ++s) {
                steps[s] = longer * (double)((k_steps + s - 1) / s);
                sums[s] = s * pieces > 1 ? (2.0 * s * pieces + 1.0) * (double)outputs * 4.0 / 8e6 : 0.0;
            }
        }
    };
    const Parts pw(has_w, (M + KSTEP - 1) / KSTEP, 1.1, 2 * F * K, pieces), px(has_x, (2 * F + KSTEP - 1) / KSTEP, 1.0, M * K, pieces);
    for (int t = 0; t <= (pieces > 1 ? kLargest - 1 : kLargest); ++t) {   // (the largest have no parts)
        const GradTile &tile = kGradTiles[t];
        auto count = [&](int64_t m, int64_t n) {
            return (double)((m + tile.bm - 1) / tile.bm) * (double)((n + tile.bn - 1) / tile.bn);
        };
        const double tiles_w = has_w ? pieces * count(2 * F, K) : 0.0, tiles_x = has_x ? pieces * count(M, K) : 0.0;
        const double limit = (double)(grid_limit(tile.threads) - kShareMore);
        for (int sw = pw.least; sw <= (t == kLargest ? pw.least : pw.most); ++sw)
            for (int sx = px.least; sx <= (t == kLargest ? px.least : px.most); ++sx) {
                const double nw = tiles_w * sw, nx = tiles_x * sx, n = nw + nx;
                if (n > limit) continue;
                const double longest = pw.steps[sw] > px.steps[sx] ? pw.steps[sw] : px.steps[sx];
                const double run = n <= 256.0 ? longest * tile.first + tile.end
                                              : tile.more * ((nw * pw.steps[sw] + nx * px.steps[sx]) * (1.0 / 256.0) + 0.5 * longest) + tile.end * (n * (1.0 / 256.0) + 0.5);
                const double us = run + (sw > 1 || sx > 1 || pieces > 1 ? 3.0 : 0.0) + pw.sums[sw] + px.sums[sx];
                if (us < best.us) best = {t, sw, sx, us};
            }
    }
    return best;
}

template <int BM, int BN, int NW, int NSTAGE>
hipError_t launch_grads_tile(const ProductArgs &dw, const ProductArgs &dx, hipStream_t stream) {
    const unsigned grid = share_grid(tiles_of(dw), tiles_of(dx));   // (of the largest tiles' halves, or more than enough)
    gated_grads_kernel<BM, BN, NW, NSTAGE><<<dim3(grid), dim3(NW * 64), 0, stream>>>(dw, dx);
    return hipGetLastError();
}

hipError_t launch_grads(ProductArgs dw, ProductArgs dx, const Plan &plan, float *parts, hipStream_t stream) {
    const GradTile &tile = kGradTiles[plan.tile];
    if (dw.splits) dw.splits = plan.parts_w;
    if (dx.splits) dx.splits = plan.parts_x;
    if (!lay_out(dw.mm, tile.bm, tile.bn, tile.threads) || !lay_out(dx.mm, tile.bm, tile.bn, tile.threads))   // (plan_of saw to it)
        return hipErrorInvalidValue;
    SumArgs sum{};
    ProductArgs *const each[2] = {&dx, &dw};
    for (int i = 0; i < 2; ++i) {
        ProductArgs &p = *each[i];
        if (p.splits * p.pieces <= 1) continue;
        const int64_t n = p.mm.M * p.mm.N;
        sum.parts[i] = parts, sum.y[i] = p.y, sum.n[i] = n, sum.bf16[i] = p.bf16, sum.splits[i] = p.splits;
        sum.pieces = p.pieces;
        p.y = parts;
        parts += p.splits * p.pieces * n;
    }
    hipError_t e = hipSuccess;
    switch (plan.tile) {
    case 0: e = launch_grads_tile<64, 64, 4, 5>(dw, dx, stream); break;
    case 1: e = launch_grads_tile<128, 128, 4, 4>(dw, dx, stream); break;
    case 2: e = launch_grads_tile<128, 256, 8, 3>(dw, dx, stream); break;
    default:
        gated_grads_large_kernel<<<dim3(share_grid(tiles_of(dw), tiles_of(dx))), dim3(512), 0, stream>>>(dw, dx);
        e = hipGetLastError();
    }
    if (e || sum.n[0] + sum.n[1] == 0) return e;
    const int64_t need = ((sum.n[0] + sum.n[1]) / 8 + 255) / 256;
    gated_sum_kernel<<<dim3((unsigned)(need < 4096 ? need : 4096)), dim3(256), 0, stream>>>(sum);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gated_linear(const uint16_t *x, const uint16_t *w, void *h, bool h_bf16, uint16_t *gu, bool gelu,
                               int64_t M, int64_t F, int64_t K, hipStream_t stream) {
    return launch_gated({{x, w, M, F, K, K, K, 0, 0, 1}, h, gu, nullptr, nullptr, gelu}, h_bf16, stream);
}

GatedGradPlans gated_gradient_plans(int64_t M, int64_t F, int64_t K, bool wide) {
    const int pieces = wide ? 2 : 1;
    GatedGradPlans p{true, true, pieces, plan_of(M, F, K, pieces, true, true), plan_of(M, F, K, pieces, true, false),
                     plan_of(M, F, K, pieces, false, true)};
    p.joint = p.both.us <= p.w.us + p.x.us + 2.0 && p.both.us < HUGE_VAL;
    p.fits = p.joint || (p.w.us < HUGE_VAL && p.x.us < HUGE_VAL);
    return p;
}

// dg and du, and their rests, then the parts' sums
size_t gated_linear_backward_workspace_bytes(const GatedGradPlans &p, int64_t M, int64_t F, int64_t K) {
    const int64_t x = p.pieces * (p.joint ? p.both.parts_x : p.x.parts_x), w = p.pieces * (p.joint ? p.both.parts_w : p.w.parts_w);
    return (size_t)(p.pieces * M * F * 4 + (x > 1 ? x * M * K * 4 : 0) + (w > 1 ? w * 2 * F * K * 4 : 0));
}

void gated_report(int64_t M, int64_t F, int64_t K, LaunchReport *r) {
    const int choice = gated_choice(M, F, K);
    if (choice >= kFew16) {
        const int nb = choice == kFew16 ? 16 : 32;
        *r = {choice == kFew32Twice ? 32 : 16, nb, 1, 0, (F + nb / 2 - 1) / (nb / 2), 256};
        return;
    }
    const GatedTile &tile = kGatedTiles[choice];
    MmArgs mm{nullptr, nullptr, M, F, K, K, K, 0, 0, 1};
    const bool fits = lay_out(mm, tile.bm, tile.bn / 2, tile.threads, choice == 4 ? kShareMore : 0);
    const int64_t tiles = (int64_t)mm.tiles_m * mm.tiles_n;
    *r = {tile.bm, tile.bn, 1, 0, !fits ? -1 : choice == 4 ? share_grid((int)tiles, 0) : tiles, tile.threads};
}

void gated_gradient_report(int64_t M, int64_t F, int64_t K, bool wide, LaunchReport *r) {
    const GatedGradPlans p = gated_gradient_plans(M, F, K, wide);
    const Plan &w = p.joint ? p.both : p.w, &x = p.joint ? p.both : p.x;
    MmArgs mw{nullptr, nullptr, 2 * F, K, M, 2 * F, K, 0, 0, 1}, mx{nullptr, nullptr, M, K, 2 * F, 2 * F, K, 0, 0, 1};
    const GradTile &tw = kGradTiles[w.tile], &tx = kGradTiles[x.tile];
    const bool fits = p.fits && lay_out(mw, tw.bm, tw.bn, tw.threads) && lay_out(mx, tx.bm, tx.bn, tx.threads);
    const int nw = fits ? mw.tiles_m * mw.tiles_n * w.parts_w * p.pieces : 0, nx = fits ? mx.tiles_m * mx.tiles_n * x.parts_x * p.pieces : 0;
    r[0] = {tw.bm, tw.bn, w.parts_w, p.joint, fits ? (int64_t)share_grid(nw, p.joint ? nx : 0) : -1, tw.threads};
    r[1] = {tx.bm, tx.bn, x.parts_x, p.joint, fits ? (int64_t)share_grid(p.joint ? nw : 0, nx) : -1, tx.threads};
}

hipError_t launch_gated_linear_backward(const uint16_t *dh, const uint16_t *x, const uint16_t *w, const uint16_t *gu,
                                        bool gelu, void *dx, bool dx_bf16, void *dw, bool dw_bf16, int64_t M, int64_t F,
                                        int64_t K, const GatedGradPlans &plans, void *workspace, hipStream_t stream) {
    uint16_t *const d = static_cast<uint16_t *>(workspace);   // [M, 2 F]
    const int64_t size = M * 2 * F;
    uint16_t *const rest = plans.pieces > 1 ? d + size : nullptr;
    float *const parts = reinterpret_cast<float *>(d + plans.pieces * size);
    if (M > 0 && F > 0) {
        if (gu) {
            const int64_t n = M * F / 8, need = (n + 255) / 256;
            const dim3 grid((unsigned)(need < 8192 ? need : 8192));
            if (rest) gated_slope_kernel<true><<<grid, dim3(256), 0, stream>>>(dh, gu, d, rest, n, F, gelu);
            else gated_slope_kernel<false><<<grid, dim3(256), 0, stream>>>(dh, gu, d, nullptr, n, F, gelu);
            if (hipError_t e = hipGetLastError()) return e;
        } else if (hipError_t e = launch_gated({{x, w, M, F, K, K, K, 0, 0, 1}, nullptr, d, dh, rest, gelu}, 2, stream)) {
            return e;
        }
    }
    const ProductArgs px{{d, w, M, K, 2 * F, 2 * F, K, 0, 0, 1}, dx, dx_bf16, dx && M > 0 && K > 0, plans.pieces, size};
    const ProductArgs pw{{d, x, 2 * F, K, M, 2 * F, K, 0, 0, 1}, dw, dw_bf16, dw && F > 0 && K > 0, plans.pieces, size};
    if (plans.joint) return px.splits || pw.splits ? launch_grads(pw, px, plans.both, parts, stream) : hipSuccess;
    // (one after the other: their parts' sums may share their place)
    ProductArgs none{};
    if (pw.splits)
        if (hipError_t e = launch_grads(pw, none, plans.w, parts, stream)) return e;
    if (px.splits)
        if (hipError_t e = launch_grads(none, px, plans.x, parts, stream)) return e;
    return hipSuccess;
}

}  // namespace fp8q
