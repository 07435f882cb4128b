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
// u keeps its 32 bits: the matrix unit takes it as three bf16 numbers whose sum it is, of which the first decides
// where B is infinite. What an adapter
// holds reaches no row of another one (not even as 0 * NaN): sums of rows with other ids are dropped.
#include <cmath>

#include <fp8q.h>

#include "mm.h"

namespace fp8q {
namespace {

constexpr int kMaxSplits = 8;   // parts of K in the adapters' first product

struct AdapterArgs {
    MmArgs mm;
    const float *bias;       // [N] or null
    const uint16_t *a, *b;   // [adapters, rank, K], [adapters, N, rank]
    const float *scales;     // [adapters] or null
    const int32_t *ids;      // [M]
    float *u;                // [splits, M, rank]
    const void *base;        // [M, N] of y's type: added instead of a product with W
    void *y;
    int adapters, rank, splits;
};

// an adapter's number, -1 where there is none
__device__ __forceinline__ int adapter_of(const AdapterArgs &g, int64_t m) {
    const int e = m < g.mm.M ? g.ids[m] : -1;
    return e >= 0 && e < g.adapters ? e : -1;
}

// u in two ways. K is cut into `splits` parts, whose sums are kept apart (u[part]) and added where u is used.
//
// Few rows, which may all have different adapters: a workgroup takes 16 ranks of one row and one part of K, its 4 waves
// a quarter of that each, A straight from memory into the matrix unit's registers, whose other operand is the row 16
// times. Bound by latency and the reads of A (250 rows of 7168 at rank 64: 34 us, 6.7 TB/s from the caches). All of a row's
// 64 ranks in one workgroup took 13.3 us at 30 rows of 3000, now 4.1.
__global__ __launch_bounds__(256) void adapter_row_kernel(AdapterArgs g) {
    constexpr int U = 4;   // steps of 64 k on their way
    __shared__ f32x4 part[4][4];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row = lane & 15, kg = lane >> 4;
    const int64_t m = blockIdx.x, K = g.mm.K;
    const int e = adapter_of(g, m), r0 = 16 * blockIdx.z, r = r0 + row;
    if (e < 0) return;
    const rsrc_t rx = make_rsrc(g.mm.x + m * K, 2 * K), ra = make_rsrc(g.a + (int64_t)e * g.rank * K, 2 * g.rank * K);
    const int steps = (int)((K + KSTEP - 1) / KSTEP), parts = 4 * g.splits, p = 4 * blockIdx.y + wave;
    const int s0 = (int)((int64_t)p * steps / parts), s1 = (int)((int64_t)(p + 1) * steps / parts);
    const uint32_t pitch = (uint32_t)(2 * K);
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    for (int s = s0; s < s1; s += U) {
        u32x4 xf[U][2], af[U][2];
#pragma unroll
        for (int v = 0; v < U; ++v)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t k = (uint32_t)((s + v) * KB + 64 * h + 16 * kg);
                const bool in = s + v < s1 && k < pitch;
                xf[v][h] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rx, in ? k : kNowhere, 0, 0));
                af[v][h] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                    ra, in && r < g.rank ? r * pitch + k : kNowhere, 0, 0));
            }
#pragma unroll
        for (int v = 0; v < U; ++v)
#pragma unroll
            for (int h = 0; h < 2; ++h) acc = mfma_bf16(af[v][h], xf[v][h], acc);
    }
    if (row == 0) part[wave][kg] = acc;
    __syncthreads();
    const int at = r0 + 4 * (int)threadIdx.x;
    if (threadIdx.x < 4 && at < g.rank) {
        f32x4 sum = part[0][threadIdx.x];
#pragma unroll
        for (int w = 1; w < 4; ++w) sum += part[w][threadIdx.x];
        const float scale = g.scales ? g.scales[e] : 1.0f;
        *reinterpret_cast<f32x4 *>(g.u + ((int64_t)blockIdx.y * g.mm.M + m) * g.rank + at) = sum * scale;
    }
}

// Many rows: tiles of 32 rows x 64 ranks (mm.h), for each of the rows' adapters, of which workgroup
// blockIdx.z takes those numbered blockIdx.z, blockIdx.z + gridDim.z, ...: mostly there is one. Bound by the copies of x
// and A into LDS, some 65 KB/us a CU (8192 x 7168 at rank 64 31-44 us for 117 MB of x, 1021 rows at 24 7.6).
using ShrinkTile = Tile<32, 64, 4, 2, 6>;
__global__ __launch_bounds__(256) void adapter_shrink_kernel(AdapterArgs g) {
    using T = ShrinkTile;
    __shared__ __attribute__((aligned(16))) uint8_t smem[T::STAGE * T::NSTAGE];
    const int lane = threadIdx.x & 63, wm = wave_m<T>(), wn = wave_n<T>();
    const int64_t m0 = (int64_t)blockIdx.x * T::BM, K = g.mm.K;
    const int steps = (int)((K + KSTEP - 1) / KSTEP), blocks = (g.rank + T::BN - 1) / T::BN;
    const int part = blockIdx.y / blocks, r0 = (blockIdx.y - part * blocks) * T::BN;
    const int64_t k0 = (int64_t)part * steps / g.splits * KSTEP, k1 = (int64_t)(part + 1) * steps / g.splits * KSTEP;
    MmArgs mm = g.mm;
    mm.x += k0;
    mm.N = g.rank;
    mm.K = (k1 < K ? k1 : K) - k0;
    const int id = lane < T::BM ? adapter_of(g, m0 + lane) : -1;
    int number = 0;
    for (uint64_t left = __ballot(id >= 0); left; ++number) {
        const int e = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        left &= ~__ballot(id == e);
        if (number % gridDim.z != blockIdx.z) continue;
        mm.w = g.a + (int64_t)e * g.rank * K + k0;
        f32x4 acc[T::SUB_M][T::SUB_N];
        multiply<T, 0, 0, 0, 2>(mm, m0, r0, smem, acc, []() {});
        const float scale = g.scales ? g.scales[e] : 1.0f;
#pragma unroll
        for (int i = 0; i < T::SUB_M; ++i) {
            const int within = T::row(wm, i) + (lane & 15);
            if (__shfl(id, within, 64) != e) continue;
#pragma unroll
            for (int j = 0; j < T::SUB_N; ++j) {
                const int r = r0 + wn * T::WN + 16 * j + 4 * (lane >> 4);
                if (r < g.rank)
                    *reinterpret_cast<f32x4 *>(g.u + ((int64_t)part * g.mm.M + m0 + within) * g.rank + r) = acc[i][j] * scale;
            }
        }
    }
}

// 32 ranks of the u of ROWS rows into LDS (fp32, pitch UP), the parts of K added in order; zeros past the rank
// and where a row has no adapter. Read by each lane for itself from memory they took longer than all
// else that an adapter costs (1021 x 1533, 8 parts: 27 us, now 7). For the whole workgroup; what reads it comes after
// a barrier.
constexpr int kChunk = 32, UP = kChunk + 4;
template <int ROWS, int THREADS>
__device__ __forceinline__ void stage_u(const AdapterArgs &g, int64_t m0, int r0, float *lds) {
    for (int p = threadIdx.x; p < ROWS * (kChunk / 4); p += THREADS) {
        const int row = p / (kChunk / 4), r = r0 + 4 * (p % (kChunk / 4));
        const int64_t m = m0 + row;
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
        if (r < g.rank && adapter_of(g, m) >= 0) {
            const float *from = g.u + m * g.rank + r;
            f32x4 part[kMaxSplits];
#pragma unroll
            for (int s = 0; s < kMaxSplits; ++s)
                part[s] = s < g.splits ? *reinterpret_cast<const f32x4 *>(from + s * g.mm.M * g.rank) : f32x4{0.f, 0.f, 0.f, 0.f};
            v = part[0];
#pragma unroll
            for (int s = 1; s < kMaxSplits; ++s) v += part[s];
        }
        *reinterpret_cast<f32x4 *>(lds + row * UP + 4 * (p % (kChunk / 4))) = v;
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
// mostly one. col: the wave's first column. For the whole workgroup.
template <class T>
__device__ __forceinline__ void add_adapters(const AdapterArgs &g, int64_t m0, int64_t col, float *lds,
                                             f32x4 (&acc)[T::SUB_M][T::SUB_N]) {
    const int lane = threadIdx.x & 63, wm = wave_m<T>(), row = lane & 15, kg = lane >> 4;
    for (int r0 = 0; r0 < g.rank; r0 += kChunk) {
        __syncthreads();
        stage_u<T::BM, T::NW * 64>(g, m0, r0, lds);
        __syncthreads();
        const int r = r0 + 8 * kg;
#pragma unroll
        for (int i = 0; i < T::SUB_M; ++i) {
            const int within = T::row(wm, i) + row;
            const int id = adapter_of(g, m0 + within);
            const float *u = lds + within * UP + 8 * kg;
            const f32x4 lo = *reinterpret_cast<const f32x4 *>(u), hi = *reinterpret_cast<const f32x4 *>(u + 4);
            u32x4 xf[3];
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                uint32_t s[2][3];
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    split3(p < 2 ? lo[2 * p + q] : hi[2 * p - 4 + q], s[q][0], s[q][1], s[q][2]);
#pragma unroll
                for (int t = 0; t < 3; ++t) xf[t][p] = s[0][t] >> 16 | s[1][t];
            }
            // AT adapters at a time, all their loads on their way together (a decode batch's 16 rows may have 16)
            for (uint64_t left = __ballot(id >= 0); left;) {
                constexpr int AT = T::SUB_M * T::SUB_N > 16 || T::NSTAGE == 1 ? 2 : 4;   // (as the registers allow)
                int e[AT];
                u32x4 wf[AT][T::SUB_N];
#pragma unroll
                for (int a = 0; a < AT; ++a) {
                    e[a] = -2;
                    if (!left) continue;
                    e[a] = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
                    left &= ~__ballot(id == e[a]);
                    const uint16_t *b = g.b + (int64_t)e[a] * g.mm.N * g.rank;
#pragma unroll
                    for (int j = 0; j < T::SUB_N; ++j) {
                        const int64_t n = col + 16 * j + row;
                        wf[a][j] = u32x4{0, 0, 0, 0};
                        if (n < g.mm.N && r < g.rank) wf[a][j] = *reinterpret_cast<const u32x4 *>(b + n * g.rank + r);
                    }
                }
#pragma unroll
                for (int a = 0; a < AT; ++a) {
                    if (e[a] == -2) continue;
#pragma unroll
                    for (int j = 0; j < T::SUB_N; ++j) {
                        const f32x4 first = mfma_bf16(wf[a][j], xf[0], f32x4{0.f, 0.f, 0.f, 0.f});
                        const f32x4 sum = mfma_bf16(wf[a][j], xf[2], mfma_bf16(wf[a][j], xf[1], first));
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            // (an infinite B times a lower number of 0 is NaN: then the first number's sum is u B's)
                            const float all = sum[q] == sum[q] ? sum[q] : first[q];
                            acc[i][j][q] = id == e[a] ? acc[i][j][q] + all : acc[i][j][q];   // (another row's -0 stays)
                        }
                    }
                }
            }
        }
    }
}

// The same where rows may all have different adapters: each lane takes its row's adapter by itself, in fp32, for
// the 4 columns of each of its blocks. begin() asks for the first 16 ranks of B and puts the first ranks of u into
// LDS; end() comes after the product, during which those loads arrive (waited for at once, they and the ids before
// them took 8 us of a 48 x 7168 x 7168 product's 30).
template <int SM, int SN, int ROWS, int THREADS>
struct OwnAdapters {
    int id[SM];
    u32x4 first[SM][SN][4][2];

    // B's ranks r .. r + 7 for columns n .. n + 3; columns past N repeat the last one (they are not stored)
    __device__ __forceinline__ void read(const AdapterArgs &g, int e, int64_t n, int r, u32x4 (&v)[4]) const {
        const uint16_t *b = g.b + ((int64_t)e * g.mm.N + n) * g.rank + r;
        const int64_t last = g.mm.N - 1 - n;
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = *reinterpret_cast<const u32x4 *>(b + (q < last ? q : last) * g.rank);
    }
    __device__ __forceinline__ static void add(const float *u, const u32x4 (&v)[4], f32x4 &sum) {
        const f32x4 lo = *reinterpret_cast<const f32x4 *>(u), hi = *reinterpret_cast<const f32x4 *>(u + 4);
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                sum[q] = __builtin_fmaf(p < 2 ? lo[2 * p] : hi[2 * p - 4], bf16lo_to_f32(v[q][p]), sum[q]);
                sum[q] = __builtin_fmaf(p < 2 ? lo[2 * p + 1] : hi[2 * p - 3], bf16hi_to_f32(v[q][p]), sum[q]);
            }
    }
    // within: the lane's row of group i, i = 0 .. SM - 1, counted from m0; col: the first of its columns in block j
    template <class W, class C>
    __device__ __forceinline__ void begin(const AdapterArgs &g, int64_t m0, float *lds, const W &within, const C &col) {
#pragma unroll
        for (int i = 0; i < SM; ++i) id[i] = adapter_of(g, m0 + within(i));
        stage_u<ROWS, THREADS>(g, m0, 0, lds);
#pragma unroll
        for (int i = 0; i < SM; ++i)
#pragma unroll
            for (int j = 0; j < SN; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (id[i] >= 0 && col(j) < g.mm.N && 8 * h < g.rank) {
                        u32x4 v[4];
                        read(g, id[i], col(j), 8 * h, v);
#pragma unroll
                        for (int q = 0; q < 4; ++q) first[i][j][q][h] = v[q];
                    }
    }
    template <class W, class C>
    __device__ __forceinline__ void end(const AdapterArgs &g, int64_t m0, float *lds, const W &within, const C &col,
                                        f32x4 (&acc)[SM][SN]) const {
        for (int r0 = 0; r0 < g.rank; r0 += kChunk) {
            if (r0) {
                __syncthreads();
                stage_u<ROWS, THREADS>(g, m0, r0, lds);
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < SM; ++i)
#pragma unroll
                for (int j = 0; j < SN; ++j) {
                    if (id[i] < 0 || col(j) >= g.mm.N) continue;
                    const float *u = lds + within(i) * UP;
#pragma unroll
                    for (int r = 0; r < kChunk; r += 8) {
                        if (r0 + r >= g.rank) continue;
                        u32x4 v[4];
                        if (r0 == 0 && r < 16) {
#pragma unroll
                            for (int q = 0; q < 4; ++q) v[q] = first[i][j][q][r / 8];
                        } else {
                            read(g, id[i], col(j), r0 + r, v);
                        }
                        add(u + r, v, acc[i][j]);
                    }
                }
        }
    }
};

__device__ __forceinline__ f32x4 bias_of(const AdapterArgs &g, int64_t n) {
    return g.bias && n < g.mm.N ? load4<0>(g.bias, n, g.mm.N - n) : f32x4{0.f, 0.f, 0.f, 0.f};
}

// A tile. ADD: no W, base is added. SHARED: rows by the matrix unit, whose neighbours mostly have one adapter, after the
// product; else each lane for itself, while the product's first copies are on their way. At rank 64 on the device:
// 8192 x 7168 x 7168 655 us, the matrix unit busy 0.65 (5000 rows 91% of the rate without adapters); added alone, 5000 x
// 7168 in runs of 90 rows 111 us (28 are the outputs' bytes at a copy's rate, the rest waits for u, ids and B in turn). A decode batch of 48 x
// 7168 x 7168 at rank 16 30 us, 3.8 TB/s: each workgroup copies all of x into its LDS at a CU's 65 KB/us.
template <class T, int SHARED>
constexpr int tile_bytes() {   // (u over the stages where it is read after the product)
    constexpr int U = 4 * UP * T::BM, STAGES = T::STAGE * T::NSTAGE;
    return SHARED ? (U > STAGES ? U : STAGES) : STAGES + U;
}
template <class T, int SHARED, int ADD, int OUT_BF16>
__device__ __forceinline__ void adapter_tile(const AdapterArgs &g, int64_t m0, int64_t n0, uint8_t *smem) {
    float *const lds = reinterpret_cast<float *>(smem + (SHARED ? 0 : T::STAGE * T::NSTAGE));
    const int lane = threadIdx.x & 63, wm = wave_m<T>(), wn = wave_n<T>();
    const int64_t col = n0 + wn * T::WN, M = g.mm.M, N = g.mm.N;
    f32x4 acc[T::SUB_M][T::SUB_N];
    auto within = [&](int i) { return T::row(wm, i) + (lane & 15); };
    auto first = [&](int j) { return col + 16 * j + 4 * (lane >> 4); };
    OwnAdapters<SHARED ? 1 : T::SUB_M, SHARED ? 1 : T::SUB_N, T::BM, T::NW * 64> own;
    auto begin = [&]() {
        if constexpr (!SHARED) own.begin(g, m0, lds, within, first);
    };
    if constexpr (ADD) {
#pragma unroll
        for (int i = 0; i < T::SUB_M; ++i)
#pragma unroll
            for (int j = 0; j < T::SUB_N; ++j) {
                const int64_t m = m0 + within(i), n = first(j);
                acc[i][j] = m < M && n < N ? load4<OUT_BF16>(g.base, m * N + n, N - n) : f32x4{0.f, 0.f, 0.f, 0.f};
            }
        begin();
    } else {
        multiply<T, 0, 0, 0, OUT_BF16>(g.mm, m0, n0, smem, acc, begin);
    }
    if constexpr (SHARED) add_adapters<T>(g, m0, col, lds, acc);
    else own.end(g, m0, lds, within, first, acc);
    f32x4 bias[T::SUB_N];
#pragma unroll
    for (int j = 0; j < T::SUB_N; ++j) bias[j] = bias_of(g, col + 16 * j + 4 * (lane >> 4));
    store_tile<T, OUT_BF16, T::SUB_N>(g.y, N, m0, M, n0, N, smem, [&](int i, int j) {
        return g.bias ? acc[i][j] + bias[j] : acc[i][j];   // (-0 + 0 would be 0)
    });
}

template <int BM, int BN, int NW, int NSTAGE, int SHARED, int ADD, int OUT_BF16>
__global__ __launch_bounds__(NW * 64) __attribute__((amdgpu_waves_per_eu(NW == 8 ? 2 : 1, 2))) void adapter_kernel(AdapterArgs g) {
    using T = Tile<BM, BN, NW, 2, NSTAGE>;
    __shared__ __attribute__((aligned(16))) uint8_t smem[tile_bytes<T, SHARED>()];
    int64_t m0, n0;
    find_tile<T, BN>(g.mm, m0, n0);
    adapter_tile<T, SHARED, ADD, OUT_BF16>(g, m0, n0, smem);
}

template <int OUT_BF16>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void adapter_large_kernel(AdapterArgs g) {
    __shared__ __attribute__((aligned(16))) uint8_t smem[tile_bytes<HalfTile, 1>()];
    static_assert(tile_bytes<HalfTile, 1>() >= tile_bytes<WholeTile, 1>(), "LDS of both");
    bool second;
    int tile, half;
    if (!find_share(g.mm.tiles_m * g.mm.tiles_n, 0, second, tile, half)) return;
    int64_t m0, n0;
    place_tile(g.mm, tile, 256, 256, m0, n0);
    if (half < 0) {
        adapter_tile<WholeTile, 1, 0, OUT_BF16>(g, m0, n0, smem);
    } else {
        m0 += 128 * half;
        if (m0 < g.mm.M) adapter_tile<HalfTile, 1, 0, OUT_BF16>(g, m0, n0, smem);
    }
}

// At most 16 rows
template <int NB, int OUT_BF16>
__global__ __launch_bounds__(256) void adapter_few_kernel(AdapterArgs g) {
    __shared__ __attribute__((aligned(16))) uint8_t smem[Few<1, NB>::BYTES];
    __shared__ __attribute__((aligned(16))) float u[16 * UP];
    const int64_t n0 = (int64_t)blockIdx.x * NB, N = g.mm.N;
    // four columns of a row a thread, 4 NB threads in all
    const int row = (threadIdx.x / (NB / 4)) & 15, at = 4 * (threadIdx.x % (NB / 4));
    const bool mine = threadIdx.x < 4 * NB;
    const int64_t n = mine ? n0 + at : N;
    auto within = [&](int) { return row; };
    auto first = [&](int) { return n; };
    OwnAdapters<1, 1, 16, 256> own;
    const float *const sums = few<1, NB, 0, OUT_BF16>(g.mm, n0, smem, [&]() { own.begin(g, 0, u, within, first); });
    f32x4 acc[1][1] = {{*reinterpret_cast<const f32x4 *>(sums + row * NB + at)}};
    own.end(g, 0, u, within, first, acc);
    if (mine && row < g.mm.M && n < N) store4<OUT_BF16>(g.y, row * N + n, g.bias ? acc[0][0] + bias_of(g, n) : acc[0][0], N - n);
}

// SHARED from 65 rows on, us at rank 64: 90 rows an adapter, 250 x 7168 x 7168 82 / 107, 500 x 3000 x 3000 41 / 61;
// one row an adapter 107 / 124 and 71 / 93, 500 x 1000 x 1000 at rank 16 15 / 14.
template <int BM, int BN, int NW, int NSTAGE, int SHARED = BM >= 128>
hipError_t launch_tile(AdapterArgs a, bool out_bf16, hipStream_t stream) {
    if constexpr (!SHARED)
        if (a.mm.M > 64) return launch_tile<BM, BN, NW, NSTAGE, 1>(a, out_bf16, stream);
    if (!lay_out(a.mm, BM, BN, NW * 64)) return hipErrorInvalidValue;
    const dim3 grid((unsigned)(a.mm.tiles_m * a.mm.tiles_n)), block(NW * 64);
    if (out_bf16) adapter_kernel<BM, BN, NW, NSTAGE, SHARED, 0, 1><<<grid, block, 0, stream>>>(a);
    else adapter_kernel<BM, BN, NW, NSTAGE, SHARED, 0, 0><<<grid, block, 0, stream>>>(a);
    return hipGetLastError();
}
hipError_t launch_large(AdapterArgs a, bool out_bf16, hipStream_t stream) {
    if (!lay_out(a.mm, 256, 256, 512, kShareMore)) return hipErrorInvalidValue;
    const dim3 grid(share_grid(a.mm.tiles_m * a.mm.tiles_n, 0)), block(512);
    if (out_bf16) adapter_large_kernel<1><<<grid, block, 0, stream>>>(a);
    else adapter_large_kernel<0><<<grid, block, 0, stream>>>(a);
    return hipGetLastError();
}
// (stages only for the room: LDS holds u and the outputs)
template <int BM, int BN, int SHARED>
hipError_t launch_add(AdapterArgs a, bool out_bf16, hipStream_t stream) {
    if (!lay_out(a.mm, BM, BN, 256)) return hipErrorInvalidValue;
    const dim3 grid((unsigned)(a.mm.tiles_m * a.mm.tiles_n)), block(256);
    if (out_bf16) adapter_kernel<BM, BN, 4, BM == 32 ? 2 : 1, SHARED, 1, 1><<<grid, block, 0, stream>>>(a);
    else adapter_kernel<BM, BN, 4, BM == 32 ? 2 : 1, SHARED, 1, 0><<<grid, block, 0, stream>>>(a);
    return hipGetLastError();
}

template <int NB>
hipError_t launch_few(const AdapterArgs &a, bool out_bf16, hipStream_t stream) {
    const dim3 grid((unsigned)((a.mm.N + NB - 1) / NB)), block(256);
    if (out_bf16) adapter_few_kernel<NB, 1><<<grid, block, 0, stream>>>(a);
    else adapter_few_kernel<NB, 0><<<grid, block, 0, stream>>>(a);
    return hipGetLastError();
}

// Whether the rows are taken one by one in the first product: A is then read for each of them (from the caches),
// which at 32 ranks of 512 rows takes as long as the tiles take with a different adapter in every row.
bool by_rows(int64_t M, int64_t rank) { return M <= 512 && M * rank <= 16384; }

// The parts of K: enough for two workgroups a CU, each with some steps to go
int splits_of(int64_t M, int64_t K, int64_t rank) {
    const int64_t steps = (K + KSTEP - 1) / KSTEP;
    const int64_t wgs = by_rows(M, rank) ? M * ((rank + 15) / 16) : (M + ShrinkTile::BM - 1) / ShrinkTile::BM * ((rank + ShrinkTile::BN - 1) / ShrinkTile::BN);
    const int64_t least = by_rows(M, rank) ? 16 : 8, most = steps / least < kMaxSplits ? steps / least : kMaxSplits;
    int64_t n = 512 / (wgs < 1 ? 1 : wgs);
    n = n < most ? n : most;
    return n < 1 ? 1 : (int)n;
}

hipError_t launch_shrink(const AdapterArgs &a, hipStream_t stream) {
    const int64_t M = a.mm.M;
    if (by_rows(M, a.rank)) {
        adapter_row_kernel<<<dim3((unsigned)M, a.splits, (a.rank + 15) / 16), dim3(256), 0, stream>>>(a);
    } else {
        const int64_t tiles = (M + ShrinkTile::BM - 1) / ShrinkTile::BM;
        const int blocks = (a.rank + ShrinkTile::BN - 1) / ShrinkTile::BN;
        // Workgroups that share a tile's adapters: 8 while that fills CUs, 2 where it only adds workgroups that find none.
        // us of both products at 7168 -> 128 with 2 / 8, in mixed order of 32 adapters and in runs of 90 rows, rank 64:
        // 520 rows (136 workgroups with 1) 76 / 58 and 15.9 / 15.8, 760 (192) 86 / 82 and 17.1 / 17.2, 900 (232) 100 / 96 and
        // 17.8 / 19.7, 1024 (256) 114 / 116 and 18.2 / 21.8, 8192 867 / 866 and 66 / 67; rank 128: 250 (128) 65 / 60 and 16.9 / 16.8,
        // 500 (256) 105 / 107 and 20.9 / 24.3.
        const dim3 grid((unsigned)tiles, a.splits * blocks, tiles * a.splits * blocks <= 192 ? 8 : 2);
        adapter_shrink_kernel<<<grid, dim3(256), 0, stream>>>(a);
    }
    return hipGetLastError();
}

// The second launch: few rows, a tile (with W), or a tile that only adds
struct AdapterTile {
    int bm, bn;
    double first, more, end;
};
constexpr AdapterTile kTiles[7] = {{32, 64, 0.155, 0.125, 1.1}, {64, 64, 0.21, 0.18, 1.4}, {128, 128, 0.45, 0.53, 5.0}, {128, 256, 0.75, 0.83, 5.7},
                                   {256, 256, 1.3, 1.5, 8.0}, {32, 32, 0.105, 0.085, 1.0}, {64, 32, 0.145, 0.12, 1.1}};
enum { kFew16 = 7, kFew32, kAddOwn, kAddNarrow, kAddWide };
int adapter_choice(int64_t M, int64_t N, int64_t K) {
    // (24 rows against the tiles, us: x 7168 x 7168 21.7 / 21.0, x 7168 x 2048 9.4 / 7.4)
    if (M <= 16) return N <= 4096 ? kFew16 : kFew32;
    int best = 4;
    double least = HUGE_VAL;
    for (int t = 0; t < 7; ++t) {
        const AdapterTile &tile = kTiles[t];
        const double us = tile_time(M, N, (K + KSTEP - 1) / KSTEP, tile.bm, tile.bn, tile.first, tile.more, tile.end, t == 4);
        if (us < least) least = us, best = t;
    }
    return best;
}
int added_choice(int64_t M, int64_t N, int64_t rank) {
    // Each lane for itself while that is little to read, us against the matrix unit with every row's adapter another
    // and with 90 rows an adapter: 500 x 1000 at rank 16 5.5 / 10.5 and 4.4 / 6.4, 250 x 1000 at 64 9.1 / 20 and
    // 6.2 / 9.5; 250 x 3000 at 64 20 / 20 and 11 / 9, 500 x 7168 at 64 74 / 53 and 35 / 19.
    if ((M <= 64 || M * N * rank <= 1 << 24) && (M + 31) / 32 * ((N + 31) / 32) <= grid_limit(256)) return kAddOwn;
    // A wide tile reads u's parts less often, us against 64 columns at rank 64: 5000 x 7168 94 / 150, 5000 x 1000
    // 23 / 27, 1500 x 3000 24 / 28; but where it leaves CUs idle: 1500 x 1000 17 / 11, 500 x 7168 55 / 57, 500 x 3000 56 / 27.
    return ((M + 63) / 64) * ((N + 255) / 256) < 256 ? kAddNarrow : kAddWide;
}

}  // namespace

size_t adapter_linear_workspace_bytes(int64_t M, int64_t K, int64_t rank) {
    return (size_t)(splits_of(M, K, rank) * M * rank * 4);
}

hipError_t launch_adapter_linear(const uint16_t *x, const uint16_t *w, const float *bias, const uint16_t *a,
                                 const uint16_t *b, const float *scales, const int32_t *ids, const void *base, void *y,
                                 bool out_bf16, int64_t M, int64_t N, int64_t K, int64_t adapters, int64_t rank,
                                 void *workspace, hipStream_t stream) {
    AdapterArgs g{{x, w, M, N, K, K, K, 0, 0, 1}, bias, a, b, scales, ids, static_cast<float *>(workspace), w ? nullptr : base, y,
                  (int)adapters, (int)rank, splits_of(M, K, rank)};
    if (adapters > 0)
        if (hipError_t e = launch_shrink(g, stream)) return e;
    switch (!w && base ? added_choice(M, N, rank) : adapter_choice(M, N, K)) {
    case kAddOwn: return launch_add<32, 32, 0>(g, out_bf16, stream);
    case kAddNarrow: return launch_add<64, 64, 1>(g, out_bf16, stream);
    case kAddWide: return launch_add<64, 256, 1>(g, out_bf16, stream);
    case kFew16: return launch_few<16>(g, out_bf16, stream);
    case kFew32: return launch_few<32>(g, out_bf16, stream);
    case 0: return launch_tile<32, 64, 4, 6>(g, out_bf16, stream);
    case 1: return launch_tile<64, 64, 4, 5>(g, out_bf16, stream);
    case 2: return launch_tile<128, 128, 4, 4>(g, out_bf16, stream);
    case 3: return launch_tile<128, 256, 8, 3>(g, out_bf16, stream);
    case 4: return launch_large(g, out_bf16, stream);
    case 5: return launch_tile<32, 32, 4, 8>(g, out_bf16, stream);
    default: return launch_tile<64, 32, 4, 8>(g, out_bf16, stream);
    }
}

void adapter_report(int64_t M, int64_t N, int64_t K, int64_t rank, bool add, LaunchReport *r) {
    const int choice = add ? added_choice(M, N, rank) : adapter_choice(M, N, K);
    const bool few = choice == kFew16 || choice == kFew32;
    const int bm = few ? 16 : choice == kAddOwn ? 32 : choice >= kAddNarrow ? 64 : kTiles[choice].bm;
    const int bn = choice == kFew16 ? 16 : few || choice == kAddOwn ? 32 : choice == kAddNarrow ? 64 : choice == kAddWide ? 256 : kTiles[choice].bn;
    const int threads = choice == 3 || choice == 4 ? 512 : 256;
    const int shared = few || choice == kAddOwn ? 0 : choice >= kAddNarrow || bm >= 128 || M > 64;
    MmArgs mm{nullptr, nullptr, M, N, K, K, K, 0, 0, 1};
    const bool fits = lay_out(mm, bm, bn, threads, choice == 4 ? kShareMore : 0);
    const int64_t tiles = (int64_t)mm.tiles_m * mm.tiles_n;
    r[0] = {bm, bn, 1, shared, !fits ? -1 : choice == 4 ? share_grid((int)tiles, 0) : tiles, threads};
    const bool rows = by_rows(M, rank);
    const int64_t blocks = (rank + ShrinkTile::BN - 1) / ShrinkTile::BN, splits = splits_of(M, K, rank);
    r[1] = rows ? LaunchReport{1, 16, splits, 1, M * splits * ((rank + 15) / 16), 256}
                : LaunchReport{ShrinkTile::BM, ShrinkTile::BN, splits, 0, (M + ShrinkTile::BM - 1) / ShrinkTile::BM * splits * blocks, 256};
}

}  // namespace fp8q
