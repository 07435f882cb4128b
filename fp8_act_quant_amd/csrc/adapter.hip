// adapter.hip -- a linear layer with a low-rank adapter of its own for every row, for gfx950:
//
//     y[m] = x[m] W^T + bias + s[e] (x[m] A[e]^T) B[e]^T,   e = ids[m]; without the last term where e is no adapter
//
// or the last term added to another projection's output. Products are bf16 with fp32 sums (mm.h).
//
// Two launches. The first gives u[m] = s[e] x[m] A[e]^T in fp32: rank products of K, a small matter but
// for reading x and A. The second is the projection, to whose sums the adapters' u B^T is added while
// they are still in registers: nothing of the output goes through memory twice, and W is read once for
// all requests. Rows of one request need not be neighbours; where they are, as in a prefill batch, 16 rows
// at a time share the products with their adapter's B.
//
// u keeps its 32 bits: the matrix unit takes it as three bf16 numbers whose sum it is. What an adapter
// holds reaches no row of another one (not even as 0 * NaN): sums of rows with other ids are dropped.
#include <cmath>

#include <fp8q.h>

#include "mm.h"

namespace fp8q {
namespace {

struct AdapterArgs {
    MmArgs mm;
    const float *bias;       // [N] or null
    const uint16_t *a, *b;   // [adapters, rank, K], [adapters, N, rank]
    const float *scales;     // [adapters] or null
    const int32_t *ids;      // [M]
    float *u;                // [M, rank]
    const void *base;        // [M, N] of y's type: added instead of a product with W
    void *y;
    int adapters, rank;
};

// an adapter's number, -1 where there is none
__device__ __forceinline__ int adapter_of(const AdapterArgs &g, int64_t m) {
    const int e = m < g.mm.M ? g.ids[m] : -1;
    return e >= 0 && e < g.adapters ? e : -1;
}

// u of 16 RG rows: WAVES waves take a part of K each, the operands straight from memory (16 bytes a lane),
// and their sums are added in LDS, in order. The rows' adapters are taken one after another, workgroup
// blockIdx.y those numbered blockIdx.y, blockIdx.y + gridDim.y, ... among them. RB blocks of 16 ranks at a time.
template <int RG, int RB, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void adapter_shrink_kernel(AdapterArgs g) {
    constexpr int U = RG + RB <= 2 ? 4 : 2;   // steps of 64 k on their way
    __shared__ f32x4 part[WAVES][RG * RB][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row = lane & 15, kg = lane >> 4;
    const int64_t m0 = (int64_t)blockIdx.x * (16 * RG), K = g.mm.K;
    const int id = lane < 16 * RG ? adapter_of(g, m0 + lane) : -1;
    const int64_t rows = g.mm.M - m0 < 16 * RG ? g.mm.M - m0 : 16 * RG;
    const rsrc_t rx = make_rsrc(g.mm.x + m0 * K, 2 * rows * K);
    const int steps = (int)((K + KSTEP - 1) / KSTEP), s0 = wave * steps / WAVES, s1 = (wave + 1) * steps / WAVES;
    const uint32_t pitch = (uint32_t)(2 * K);
    int number = 0;
    for (uint64_t left = __ballot(id >= 0); left; ++number) {
        const int e = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        left &= ~__ballot(id == e);
        if (number % gridDim.y != blockIdx.y) continue;
        const rsrc_t ra = make_rsrc(g.a + (int64_t)e * g.rank * K, 2 * g.rank * K);
        for (int r0 = 0; r0 < g.rank; r0 += 16 * RB) {
            f32x4 acc[RG][RB];
#pragma unroll
            for (int i = 0; i < RG; ++i)
#pragma unroll
                for (int j = 0; j < RB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
            for (int s = s0; s < s1; s += U) {
                u32x4 xf[U][2][RG], af[U][2][RB];
#pragma unroll
                for (int v = 0; v < U; ++v)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t k = (uint32_t)((s + v) * KB + 64 * h + 16 * kg);
                        const bool in = s + v < s1 && k < pitch;
#pragma unroll
                        for (int i = 0; i < RG; ++i)
                            xf[v][h][i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                rx, in ? (16 * i + row) * pitch + k : kNowhere, 0, 0));
#pragma unroll
                        for (int j = 0; j < RB; ++j)
                            af[v][h][j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                ra, in && r0 + 16 * j + row < g.rank ? (r0 + 16 * j + row) * pitch + k : kNowhere, 0, 0));
                    }
#pragma unroll
                for (int v = 0; v < U; ++v)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int i = 0; i < RG; ++i)
#pragma unroll
                            for (int j = 0; j < RB; ++j) acc[i][j] = mfma_bf16(af[v][h][j], xf[v][h][i], acc[i][j]);
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < RG; ++i)
#pragma unroll
                for (int j = 0; j < RB; ++j) part[wave][i * RB + j][lane] = acc[i][j];
            __syncthreads();
            const float scale = g.scales ? g.scales[e] : 1.0f;
            for (int b = wave; b < RG * RB; b += WAVES) {
                f32x4 sum = part[0][b][lane];
#pragma unroll
                for (int w = 1; w < WAVES; ++w) sum += part[w][b][lane];
                const int within = 16 * (b / RB) + row, r = r0 + 16 * (b % RB) + 4 * kg;
                if (__shfl(id, within, 64) == e && r < g.rank)
                    *reinterpret_cast<f32x4 *>(g.u + (m0 + within) * g.rank + r) = sum * scale;
            }
        }
    }
}

// Three bf16 numbers whose sum is v: two cut off (exactly, whatever v is) and the rest, which has 8 bits.
// Infinities and NaN are the first number's alone.
__device__ __forceinline__ void split3(float v, uint32_t &a, uint32_t &b, uint32_t &c) {
    const uint32_t bits = __float_as_uint(v);
    const bool special = (bits & 0x7F800000u) == 0x7F800000u;
    a = bits & 0xFFFF0000u;
    if (special && (bits & 0x007FFFFFu)) a = 0x7FC00000u;
    const float r = special ? 0.0f : v - __uint_as_float(a);
    b = __float_as_uint(r) & 0xFFFF0000u;
    c = __float_as_uint(r - __uint_as_float(b)) & 0xFFFF0000u;
}

// Adds the adapters' part to a wave's sums by the matrix unit: each 16-row group's adapters one after another,
// mostly one. col: the wave's first column.
template <class T>
__device__ __forceinline__ void add_adapters(const AdapterArgs &g, int64_t m0, int64_t col, f32x4 (&acc)[T::SUB_M][T::SUB_N]) {
    const int lane = threadIdx.x & 63, wm = wave_m<T>(), row = lane & 15, kg = lane >> 4;
#pragma unroll
    for (int i = 0; i < T::SUB_M; ++i) {
        const int64_t m = m0 + T::row(wm, i) + row;
        const int id = adapter_of(g, m);
        for (uint64_t left = __ballot(id >= 0); left;) {
            const int e = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
            left &= ~__ballot(id == e);
            const uint16_t *b = g.b + (int64_t)e * g.mm.N * g.rank;
            f32x4 sum[T::SUB_N];
#pragma unroll
            for (int j = 0; j < T::SUB_N; ++j) sum[j] = f32x4{0.f, 0.f, 0.f, 0.f};
            for (int r0 = 0; r0 < g.rank; r0 += 32) {
                const int r = r0 + 8 * kg;
                f32x4 lo = {0.f, 0.f, 0.f, 0.f}, hi = lo;
                if (id == e && r < g.rank) {
                    lo = *reinterpret_cast<const f32x4 *>(g.u + m * g.rank + r);
                    hi = *reinterpret_cast<const f32x4 *>(g.u + m * g.rank + r + 4);
                }
                u32x4 wf[T::SUB_N], xf[3];
#pragma unroll
                for (int j = 0; j < T::SUB_N; ++j) {
                    const int64_t n = col + 16 * j + row;
                    wf[j] = u32x4{0, 0, 0, 0};
                    if (n < g.mm.N && r < g.rank) wf[j] = *reinterpret_cast<const u32x4 *>(b + n * g.rank + r);
                }
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    uint32_t s[2][3];
#pragma unroll
                    for (int q = 0; q < 2; ++q)
                        split3(p < 2 ? lo[2 * p + q] : hi[2 * p - 4 + q], s[q][0], s[q][1], s[q][2]);
#pragma unroll
                    for (int t = 0; t < 3; ++t) xf[t][p] = s[0][t] >> 16 | s[1][t];
                }
#pragma unroll
                for (int t = 0; t < 3; ++t)
#pragma unroll
                    for (int j = 0; j < T::SUB_N; ++j) sum[j] = mfma_bf16(wf[j], xf[t], sum[j]);
            }
#pragma unroll
            for (int j = 0; j < T::SUB_N; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[i][j][q] += id == e ? sum[j][q] : 0.0f;
        }
    }
}

// The same for one 16 x 16 block whose rows may all have different adapters: each lane takes its row's
// adapter by itself, in fp32. n: the first of the lane's 4 columns.
__device__ __forceinline__ f32x4 own_adapter(const AdapterArgs &g, int64_t m, int64_t n) {
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    const int id = adapter_of(g, m);
    if (id < 0 || n >= g.mm.N) return sum;
    const float *u = g.u + m * g.rank;
    const uint16_t *b = g.b + ((int64_t)id * g.mm.N + n) * g.rank;
    const int64_t last = g.mm.N - 1 - n;
    for (int r = 0; r < g.rank; r += 8) {
        const f32x4 lo = *reinterpret_cast<const f32x4 *>(u + r), hi = *reinterpret_cast<const f32x4 *>(u + r + 4);
#pragma unroll
        for (int q = 0; q < 4; ++q) {   // (columns past N repeat the last one: they are not stored)
            const u32x4 v = *reinterpret_cast<const u32x4 *>(b + (q < last ? q : last) * g.rank + r);
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                sum[q] = __builtin_fmaf(p < 2 ? lo[2 * p] : hi[2 * p - 4], bf16lo_to_f32(v[p]), sum[q]);
                sum[q] = __builtin_fmaf(p < 2 ? lo[2 * p + 1] : hi[2 * p - 3], bf16hi_to_f32(v[p]), sum[q]);
            }
        }
    }
    return sum;
}

__device__ __forceinline__ f32x4 bias_of(const AdapterArgs &g, int64_t n) {
    return g.bias && n < g.mm.N ? load4<0>(g.bias, n, g.mm.N - n) : f32x4{0.f, 0.f, 0.f, 0.f};
}

// ADD: no W, base is added
template <int BM, int BN, int NW, int NSTAGE, int ADD, int OUT_BF16>
__global__ __launch_bounds__(NW * 64) __attribute__((amdgpu_waves_per_eu(NW == 8 ? 2 : 1, 2))) void adapter_kernel(AdapterArgs g) {
    using T = Tile<BM, BN, NW, 2, NSTAGE>;
    __shared__ __attribute__((aligned(16))) uint8_t smem[T::STAGE * NSTAGE];
    int64_t m0, n0;
    find_tile<T, BN>(g.mm, m0, n0);
    f32x4 acc[T::SUB_M][T::SUB_N];
    if constexpr (ADD) {
#pragma unroll
        for (int i = 0; i < T::SUB_M; ++i)
#pragma unroll
            for (int j = 0; j < T::SUB_N; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    } else {
        multiply<T, 0, 0, 0, OUT_BF16>(g.mm, m0, n0, smem, acc);
    }
    const int lane = threadIdx.x & 63, wm = wave_m<T>(), wn = wave_n<T>();
    const int64_t col = n0 + wn * T::WN, M = g.mm.M, N = g.mm.N;
    constexpr bool SHARED = T::SUB_M * T::SUB_N > 4;
    if constexpr (SHARED) add_adapters<T>(g, m0, col, acc);
    f32x4 bias[T::SUB_N];
#pragma unroll
    for (int j = 0; j < T::SUB_N; ++j) bias[j] = bias_of(g, col + 16 * j + 4 * (lane >> 4));
    store_tile<T, OUT_BF16, T::SUB_N>(g.y, N, m0, M, n0, N, smem, [&](int i, int j) {
        const int64_t m = m0 + T::row(wm, i) + (lane & 15), n = col + 16 * j + 4 * (lane >> 4);
        f32x4 v = acc[i][j] + bias[j];
        if constexpr (!SHARED) v += own_adapter(g, m, n);
        if constexpr (ADD) {
            if (m < M && n < N) v += load4<OUT_BF16>(g.base, m * N + n, N - n);
        }
        return v;
    });
}

template <int OUT_BF16>
__global__ __launch_bounds__(256) void adapter_few_kernel(AdapterArgs g) {
    __shared__ __attribute__((aligned(16))) uint8_t smem[kFewStage * kFewStages];
    __shared__ f32x4 part[2][64];
    const int64_t n0 = (int64_t)blockIdx.x * kFewN;
    const f32x4 acc = few<0, OUT_BF16>(g.mm, n0, smem, part);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t m = lane & 15, n = n0 + 16 * wave + 4 * (lane >> 4), N = g.mm.N;
    if (wave >= 2 || m >= g.mm.M || n >= N) return;
    store4<OUT_BF16>(g.y, m * N + n, acc + bias_of(g, n) + own_adapter(g, m, n), N - n);
}

template <int BM, int BN, int NW, int NSTAGE>
hipError_t launch_tile(AdapterArgs a, bool out_bf16, hipStream_t stream) {
    if (!lay_out(a.mm, BM, BN, NW * 64)) return hipErrorInvalidValue;
    const dim3 grid((unsigned)(a.mm.tiles_m * a.mm.tiles_n)), block(NW * 64);
    if (a.base) {
        if (out_bf16) adapter_kernel<BM, BN, NW, NSTAGE, 1, 1><<<grid, block, 0, stream>>>(a);
        else adapter_kernel<BM, BN, NW, NSTAGE, 1, 0><<<grid, block, 0, stream>>>(a);
    } else {
        if (out_bf16) adapter_kernel<BM, BN, NW, NSTAGE, 0, 1><<<grid, block, 0, stream>>>(a);
        else adapter_kernel<BM, BN, NW, NSTAGE, 0, 0><<<grid, block, 0, stream>>>(a);
    }
    return hipGetLastError();
}

hipError_t launch_shrink(const AdapterArgs &a, hipStream_t stream) {
    const int64_t M = a.mm.M;
    if (M <= 256) {
        const dim3 grid((unsigned)((M + 15) / 16), M < 16 ? (unsigned)M : 16);
        adapter_shrink_kernel<1, 1, 16><<<grid, dim3(1024), 0, stream>>>(a);
    } else if (a.rank <= 16) {
        adapter_shrink_kernel<2, 1, 8><<<dim3((unsigned)((M + 31) / 32), 2), dim3(512), 0, stream>>>(a);
    } else {
        adapter_shrink_kernel<2, 4, 8><<<dim3((unsigned)((M + 31) / 32), 2), dim3(512), 0, stream>>>(a);
    }
    return hipGetLastError();
}

}  // namespace

size_t adapter_linear_workspace_bytes(int64_t M, int64_t rank) { return (size_t)(M * rank * 4); }

hipError_t launch_adapter_linear(const uint16_t *x, const uint16_t *w, const float *bias, const uint16_t *a,
                                 const uint16_t *b, const float *scales, const int32_t *ids, const void *base, void *y,
                                 bool out_bf16, int64_t M, int64_t N, int64_t K, int64_t adapters, int64_t rank,
                                 void *workspace, hipStream_t stream) {
    AdapterArgs g{{x, w, M, N, K, K, K, 0, 0, 1}, bias, a, b, scales, ids, static_cast<float *>(workspace), w ? nullptr : base, y,
                  (int)adapters, (int)rank};
    if (adapters > 0)
        if (hipError_t e = launch_shrink(g, stream)) return e;
    if (!w) return M <= 256 ? launch_tile<32, 64, 4, 6>(g, out_bf16, stream) : launch_tile<128, 128, 4, 4>(g, out_bf16, stream);
    if (M <= kFewRows) {
        const dim3 grid((unsigned)((N + kFewN - 1) / kFewN)), block(256);
        if (out_bf16) adapter_few_kernel<1><<<grid, block, 0, stream>>>(g);
        else adapter_few_kernel<0><<<grid, block, 0, stream>>>(g);
        return hipGetLastError();
    }
    auto time = [&](int bm, int bn, double first, double more, double end) {
        const double tiles = (double)((M + bm - 1) / bm) * (double)((N + bn - 1) / bn), rounds = std::ceil(tiles / 256.0);
        return (double)((K + KSTEP - 1) / KSTEP) * (first + more * (rounds - 1.0)) + end * rounds;
    };
    const double t[5] = {time(32, 64, 0.155, 0.125, 1.1), time(64, 64, 0.21, 0.18, 1.4), time(128, 128, 0.45, 0.53, 5.0),
                         time(128, 256, 0.75, 0.83, 5.7), time(256, 256, 1.3, 1.5, 8.0)};
    int best = 0;
    for (int i = 1; i < 5; ++i)
        if (t[i] < t[best]) best = i;
    switch (best) {
    case 0: return launch_tile<32, 64, 4, 6>(g, out_bf16, stream);
    case 1: return launch_tile<64, 64, 4, 5>(g, out_bf16, stream);
    case 2: return launch_tile<128, 128, 4, 4>(g, out_bf16, stream);
    case 3: return launch_tile<128, 256, 8, 3>(g, out_bf16, stream);
    default: return launch_tile<256, 256, 8, 2>(g, out_bf16, stream);
    }
}

}  // namespace fp8q
