// int8.hip -- products in 8-bit integers with one scale per token and one per output channel,
// for gfx950, and the quantisation of rows that they take.
//
//     s[m] = RN_fp32(max |x[m, :]| * RN_fp32(1 / 127)),  q[m, k] = RNE(RN_fp32(x[m, k] / s[m]))
//     y[m, n] = RN_out(float(sum_k a[m, k] * w[n, k]) * sa[m] * sw[n] + bias[n])
//
// The sum is exact: 32-bit integers, K < 2^17, so it does not depend on tiles, splits or order.
// Only the conversion of the sum, the two scalings and the bias round, each once, in fp32.
//
// Orientation. W rows are the MFMA's A operand and token rows its B operand: lane l of a 16x16
// result holds n = 4 * (l / 16) + r (r = 0..3) for m = l % 16, four consecutive outputs of a
// row of Y. v_mfma_i32_16x16x64_i8 contracts 64 bytes of K: lane l supplies row l % 16 and the
// 16 bytes at 16 * (l / 16), the same in both operands.
//
// Grouped products. Expert e owns the rows offsets[e] .. offsets[e + 1] - 1 of Y; row r's
// token is rows[r] (the gather is part of the loads, a token is quantised once however many
// experts take it), or r itself.
#include <cmath>
#include <type_traits>

#include <fp8q.h>

#include "device_common.h"
#include "launch.h"

namespace fp8q {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __amdgpu_buffer_rsrc_t rsrc_t;

// ---- row quantisation ------------------------------------------------------------------

// A row's scale and what its codes are formed with. RN(x / s) comes from the rounded reciprocal
// and two corrections (fast_quotient's steps, of which only the sign of a zero is left out); that
// it gives the same code as the division is tested for every pair of significands of x and maximum,
// at 23 of the maximum's exponents (the significands decide while nothing leaves the normal range). It
// needs s >= 2^-92, on both sides of which those exponents lie; smaller scales take the division, and a
// clamp, since a scale below the normal range may be off by more than the half step that separates
// 127 from 127.5.
struct RowScale {
    float s, d, y;
    bool fast;
};
__device__ __forceinline__ RowScale row_scale(uint32_t top_bits) {
    RowScale r;
    r.s = __uint_as_float(top_bits << 16) * (1.0f / 127.0f);
    r.d = top_bits ? r.s : 1.0f;
    r.y = 1.0f / r.d;
    r.fast = r.d >= kFastDivMin;
    return r;
}

// 8 codes of 8 bf16 values. Adding 1.5 * 2^23 rounds to the nearest whole number, ties to even, and
// leaves it in the low bits.
__device__ __forceinline__ u32x2 codes8(u32x4 v, const RowScale &r) {
    u32x2 out;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t c[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const uint32_t u = v[2 * h + b / 2];
            const float x = b & 1 ? bf16hi_to_f32(u) : bf16lo_to_f32(u);
            const float q0 = x * r.y;
            float q = __builtin_fmaf(__builtin_fmaf(-q0, r.d, x), r.y, q0);
            if (!r.fast) q = __builtin_amdgcn_fmed3f(x / r.d, -127.0f, 127.0f);
            c[b] = __float_as_uint(q + 0x1.8p23f);
        }
        const uint32_t lo = __builtin_amdgcn_perm(c[1], c[0], 0x0C0C0400);   // bytes 0 of c[0], c[1]
        const uint32_t hi = __builtin_amdgcn_perm(c[3], c[2], 0x04000C0C);   // of c[2], c[3], above
        out[h] = lo | hi;
    }
    return out;
}

__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
    v = row16_max(v);
#pragma unroll
    for (int m = 16; m < 64; m <<= 1) {
        const uint32_t o = __shfl_xor(v, m, 64);
        v = v > o ? v : o;
    }
    return v;
}

// Bound by memory: 16384 x 7168 54 us, 6.5 TB/s. WAVES waves to a row, which they keep in registers
// between the maximum and the codes where it has at most 512 * WAVES * NV elements (NV > 0), and read
// a second time where it is longer.
template <int WAVES, int NV>
__global__ __launch_bounds__(WAVES > 4 ? 64 * WAVES : 256) void row_quant_kernel(const uint16_t *x, int8_t *q, float *s, int64_t M, int64_t K) {
    constexpr int ROWS = WAVES > 4 ? 1 : 4 / WAVES, NT = 64 * WAVES, KEEP = NV > 0 ? NV : 1;
    __shared__ uint32_t part[WAVES > 4 ? WAVES : 4];
    const int tid = threadIdx.x % NT;
    const int64_t m = (int64_t)blockIdx.x * ROWS + threadIdx.x / NT;
    const bool in = m < M;
    const u32x4 *src = reinterpret_cast<const u32x4 *>(x + (in ? m : 0) * K);
    const int64_t n = in ? K / 8 : 0;
    u32x4 v[KEEP];
    uint32_t top = 0;
    if constexpr (NV > 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            v[i] = u32x4{0, 0, 0, 0};
            if (tid + i * NT < n) v[i] = src[tid + i * NT];
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const uint32_t b = absmax_bits8(v[i]);
            top = top > b ? top : b;
        }
    } else {
        for (int64_t i = tid; i < n; i += NT) {
            const uint32_t b = absmax_bits8(src[i]);
            top = top > b ? top : b;
        }
    }
    top = wave_umax(top);
    if constexpr (WAVES > 1) {
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < WAVES; ++w) top = top > part[w] ? top : part[w];
    }
    const RowScale r = row_scale(top);
    u32x2 *dst = reinterpret_cast<u32x2 *>(q + (in ? m : 0) * K);
    if constexpr (NV > 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (tid + i * NT < n) dst[tid + i * NT] = codes8(v[i], r);
    } else {
        for (int64_t i = tid; i < n; i += NT) dst[i] = codes8(src[i], r);
    }
    if (in && tid == 0) s[m] = r.s;
}

// ---- products --------------------------------------------------------------------------

constexpr int KB = 128;   // bytes of K in a stage row

struct Int8Args {
    const int8_t *a;
    const float *sa;
    const int8_t *w;
    const float *sw;
    const float *bias;        // [N] or null
    void *y;
    const int64_t *offsets;   // grouped: [experts + 1]; else null
    const int32_t *rows;      // grouped: row r's token, or null (r itself)
    int64_t M, N, K;          // rows of Y, channels, depth
    int64_t tokens;           // rows of a
    int experts;
    int tiles_m, tiles_n, group;
    bool stream;              // grouped: W is larger than the last-level cache
};

constexpr int kNonTemporal = 2;   // cache policy of buffer loads
constexpr int64_t kLastLevelCache = 256 << 20;   // bytes

// A past-the-end offset: loads there return zero (every buffer here is shorter)
constexpr uint32_t kNowhere = 0xFFFFFFF0u;

__device__ __forceinline__ rsrc_t make_rsrc(const void *p, int64_t bytes) {
    const uint32_t n = bytes > (int64_t)kNowhere ? kNowhere : (uint32_t)bytes;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, (int)n, 0x00020000);
}

// 16-byte chunk c of LDS row r lies at physical chunk c ^ (r & 7): fragment reads (16 rows x 4
// chunks an instruction) then meet no bank conflict
__device__ __forceinline__ int swz_chunk(int row, int chunk) { return chunk ^ (row & 7); }

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}

__device__ __forceinline__ void lds_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

__device__ __forceinline__ i32x4 mfma_i8(const u32x4 &w, const u32x4 &x, i32x4 acc) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, w), __builtin_bit_cast(i32x4, x), acc, 0,
                                                 0, 0);
}

// An expert's rows, clamped to [0, M): nothing outside Y is touched whatever the offsets say
__device__ __forceinline__ void expert_rows(const Int8Args &g, int e, int64_t &r0, int64_t &r1) {
    r0 = g.offsets[e];
    r1 = g.offsets[e + 1];
    r0 = r0 < 0 ? 0 : (r0 > g.M ? g.M : r0);
    r1 = r1 < r0 ? r0 : (r1 > g.M ? g.M : r1);
}

// Grouped work order. An expert's rows are cut into blocks of BM, the last of them short. Its tiles
// are numbered with the row block varying fastest, experts one after another: neighbours then
// read the same weight panel, and an expert's rows stay in the L2 of the XCD that walks it. The
// numbers are dealt to the XCDs in contiguous, equal runs. (64 experts' 4096 x 7168, 12288 rows, before
// the non-temporal accesses: 508 us; numbered by size, long tiles first, 542, an expert's blocks then
// being read through several XCDs; runs of equal cost instead of equal counts 536, the grid's larger
// bound costing more than the balance gains.)
//
// Each wave works this out by itself, 64 experts at a time.
__device__ __forceinline__ int wave_scan(int v) {   // inclusive prefix sum over the lanes
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);    // row_shr 1, 2, 4, 8
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);   // row_bcast15 into rows 1 and 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);   // row_bcast31 into rows 2 and 3
    return v;
}
template <int BM>
__device__ __forceinline__ int blocks_of(const Int8Args &g, int e) {   // of expert e's rows
    int64_t r0 = 0, r1 = 0;
    if (e < g.experts) expert_rows(g, e, r0, r1);
    return ((int)(r1 - r0) + BM - 1) / BM;
}
template <int BM>
__device__ __forceinline__ int count_blocks(const Int8Args &g) {
    const int lane = threadIdx.x & 63;
    int n = 0;
    for (int e0 = 0; e0 < g.experts; e0 += 64) n += blocks_of<BM>(g, e0 + lane);
    return __builtin_amdgcn_readlane(wave_scan(n), 63);
}
// the expert, rows and column of tile `index`, and the expert's row blocks; false: there is none
template <int BM>
__device__ __forceinline__ bool find_block(const Int8Args &g, int cols, int index, int &expert, int64_t &row0,
                                           int64_t &row1, int &col, int &per) {
    const int lane = threadIdx.x & 63;
    int before = 0;
    for (int e0 = 0; e0 < g.experts; e0 += 64) {
        const int n = blocks_of<BM>(g, e0 + lane), sum = wave_scan(n), first = (before + sum - n) * cols;
        const uint64_t hit = __ballot(index >= first && index < first + n * cols);
        if (hit) {
            const int l = __builtin_ctzll(hit);
            const int within = index - __builtin_amdgcn_readlane(first, l);
            per = __builtin_amdgcn_readlane(n, l);
            expert = e0 + l;
            col = within / per;
            expert_rows(g, expert, row0, row1);
            row0 += (int64_t)(within - col * per) * BM;
            return true;
        }
        before += __builtin_amdgcn_readlane(sum, 63);
    }
    return false;
}

// Output rows start anywhere that 4 bytes (or with an odd N 2) allow; the vector stores take that
typedef u32x4 __attribute__((aligned(2))) u32x4_any;
typedef u32x2 __attribute__((aligned(2))) u32x2_any;

// four consecutive outputs of a row with `left` elements from here on
template <int OUT_BF16>
__device__ __forceinline__ void store4(void *y, int64_t at, const f32x4 &v, int64_t left) {
    if constexpr (OUT_BF16) {
        uint16_t *p = reinterpret_cast<uint16_t *>(y) + at;
        const u32x2 u = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        if (left >= 4) {
            *reinterpret_cast<u32x2_any *>(p) = u;
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (r < left) p[r] = (uint16_t)(u[r / 2] >> (16 * (r & 1)));
        }
    } else {
        float *p = reinterpret_cast<float *>(y) + at;
        if (left >= 4) {
            *reinterpret_cast<u32x4_any *>(p) = __builtin_bit_cast(u32x4, v);
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (r < left) p[r] = v[r];
        }
    }
}

// At most 8 rows (a decode step): every byte of W meets all of them once, so the read of W is
// what counts. A workgroup takes 16 channels; its 4 waves take a quarter of K each, W straight
// from memory into MFMA operands (nothing of it is used twice), 2 U steps of 64 bytes in flight.
// The quarters are added in LDS, exactly.
//
// QUANT: the rows, of at most 2048 elements, come as bf16 and are quantised here: every workgroup does
// it for itself, in LDS, a row by a wave, while its first reads of W are on their way, which costs less
// than a launch of its own. 1 x 4096 x 2048 4.0 us, of which 3 are the launch; 8 rows 5.6.
constexpr int kFewRows = 8, kFewQuantK = 2048;

struct Int8FewArgs {
    const int8_t *a;       // QUANT: null
    const float *sa;
    const uint16_t *x;     // QUANT: [M, K] bf16
    const int8_t *w;
    const float *sw;
    const float *bias;
    void *y;
    int64_t N;
    int M, K;
};

template <int U, int QUANT, int OUT_BF16>
__global__ __launch_bounds__(256) void int8_few_kernel(Int8FewArgs g) {
    constexpr int PITCH = kFewQuantK + 16;
    __shared__ i32x4 part[4][64];
    __shared__ __attribute__((aligned(16))) uint8_t codes[QUANT ? kFewRows * PITCH : 16];
    __shared__ uint32_t tops[kFewRows];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row = lane & 15, kg = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int K = g.K, M = g.M;
    const int nw = (int)(g.N - n0 < 16 ? g.N - n0 : 16);
    const rsrc_t rw = make_rsrc(g.w + n0 * K, (int64_t)nw * K);
    const rsrc_t ra = make_rsrc(QUANT ? (const void *)g.x : g.a, QUANT ? (int64_t)M * K * 2 : (int64_t)M * K);
    const int steps = (K + 63) / 64;
    const int s0 = wave * steps / 4, s1 = (wave + 1) * steps / 4;

    i32x4 acc = {0, 0, 0, 0};
    u32x4 wv[2][U], av[2][QUANT ? 1 : U];
    // Bytes of W past K or past the last channel read as zero, which makes what the rows hold
    // there count for nothing.
    auto load = [&](int b, int s) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = (s + u) * 64 + kg * 16;
            const bool in = s + u < s1 && k < K;
            wv[b][u] = __builtin_bit_cast(
                u32x4, __builtin_amdgcn_raw_buffer_load_b128(rw, in ? (uint32_t)(row * K + k) : kNowhere, 0, 0));
            if constexpr (!QUANT)
                av[b][u] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                         ra, in && row < M ? (uint32_t)(row * K + k) : kNowhere, 0, 0));
        }
    };
    auto multiply = [&](int b, int s) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            u32x4 x = {0, 0, 0, 0};
            if constexpr (QUANT) {
                // (past K: whatever lies there, against zeros of W; always inside `codes`)
                const int k = min((s + u) * 64 + kg * 16, kFewQuantK);
                if (row < M) x = *reinterpret_cast<const u32x4 *>(codes + row * PITCH + k);
            } else {
                x = av[b][u];
            }
            acc = mfma_i8(wv[b][u], x, acc);
        }
    };
    float scale = 0.0f;   // of this lane's row
    if constexpr (QUANT) {
        constexpr int ROWS = kFewRows / 4, NV = kFewQuantK / 512;   // of a wave: every fourth row
        u32x4 v[ROWS][NV];
        // the rows first: loads return in order, and these are needed before W
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            const int m = wave + 4 * j;
            if (m < M) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int p = lane + 64 * i;
                    v[j][i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                            ra, 8 * p < K ? (uint32_t)(2 * (m * K + 8 * p)) : kNowhere, 0, 0));
                }
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        load(0, s0);
        load(1, s0 + U);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            const int m = wave + 4 * j;
            if (m < M) {
                uint32_t top = 0;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const uint32_t b = absmax_bits8(v[j][i]);
                    top = top > b ? top : b;
                }
                top = wave_umax(top);
                if (lane == 0) tops[m] = top;
                const RowScale r = row_scale(top);
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int p = lane + 64 * i;
                    if (8 * p < K) *reinterpret_cast<u32x2 *>(codes + m * PITCH + 8 * p) = codes8(v[j][i], r);
                }
            }
        }
        __syncthreads();
        if (row < M) scale = row_scale(tops[row]).s;
    } else {
        load(0, s0);
        if (row < M && K > 0) scale = g.sa[row];
    }
    for (int s = s0; s < s1; s += 2 * U) {
        if (!QUANT || s != s0) load(1, s + U);
        multiply(0, s);
        load(0, s + 2 * U);
        multiply(1, s + U);
    }

    part[wave][lane] = acc;
    __syncthreads();
    const int64_t n = n0 + 4 * kg;
    if (wave != 0 || row >= M || n >= g.N) return;
    i32x4 sum = part[0][lane];
#pragma unroll
    for (int v = 1; v < 4; ++v) sum += part[v][lane];
    f32x4 out;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int64_t nr = n + r < g.N ? n + r : g.N - 1;
        out[r] = (float)sum[r] * scale * (K > 0 ? g.sw[nr] : 0.0f) + (g.bias ? g.bias[nr] : 0.0f);
    }
    store4<OUT_BF16>(g.y, row * g.N + n, out, g.N - n);
}

// Many rows: tiles of BM x BN in LDS, NW waves in a WAVES_M x (NW / WAVES_M) grid. Tile rows go to
// the waves in groups of 16 in turn, so that a tile with fewer rows is shared evenly, and of 256 rows
// the first 128 are every wave's first half: group i of the waves in row wm of the grid starts at tile
// row row(wm, i).
template <int BM_, int BN_, int NW_, int WAVES_M_, int NSTAGE_>
struct Int8Tile {
    static constexpr int BM = BM_, BN = BN_, NW = NW_, WAVES_M = WAVES_M_, WAVES_N = NW_ / WAVES_M_;
    static constexpr int NSTAGE = NSTAGE_;
    static constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N;
    static constexpr int SUB_M = WM / 16, SUB_N = WN / 16;
    static constexpr int A_BYTES = BM * KB, W_BYTES = BN * KB, STAGE = A_BYTES + W_BYTES;
    static constexpr int A_INSTR = BM / (8 * NW), W_INSTR = BN / (8 * NW), IPW = A_INSTR + W_INSTR;
    static_assert(WAVES_M * WAVES_N == NW && BM % (8 * NW) == 0 && BN % (8 * NW) == 0, "tile shape");
    static_assert(STAGE * NSTAGE <= 160 * 1024 && IPW * (NSTAGE - 1) < 64, "LDS budget, vmcnt range");
    __device__ static __forceinline__ constexpr int row(int wm, int i) { return 16 * (i * WAVES_M + wm); }
};

// A workgroup's tile
struct TileAt {
    int64_t m0, m1, n0;   // first row, end of the rows (not of the tile), first channel
    const int8_t *w;      // the tile's weight and its scales
    const float *sw;
    // Its W panel is read once in this call, and is gone from the caches by the next one: copied
    // non-temporally (64 experts' 4096 x 7168 at 1.5 rows 203 -> 177 us; a W that stays in the caches
    // 11.0 -> 16.5, and one read by two row blocks 512 -> 560: neither is)
    bool stream;
};

// Tile of a workgroup. Workgroup b runs on XCD b % 8, and each XCD takes a contiguous run of the
// tile numbers. One weight's tiles are numbered down `group` tile rows per tile column, so that
// the tiles that an XCD holds at once share A and W panels in its L2. False: no tile (grouped: the
// grid is an upper bound).
template <class T, int GROUPED>
__device__ __forceinline__ bool find_tile(const Int8Args &g, TileAt &t) {
    const int tiles = (GROUPED ? count_blocks<T::BM>(g) : g.tiles_m) * g.tiles_n;
    const int xcd = blockIdx.x & 7, slot = blockIdx.x >> 3;
    const int q = tiles >> 3, rem = tiles & 7;
    const int tl = xcd * q + (xcd < rem ? xcd : rem) + slot;
    t.w = g.w;
    t.sw = g.sw;
    t.stream = false;
    if constexpr (GROUPED) {
        int expert, col, per;
        if (slot >= q + (xcd < rem) || !find_block<T::BM>(g, g.tiles_n, tl, expert, t.m0, t.m1, col, per)) return false;
        t.stream = g.stream && per == 1;
        t.n0 = (int64_t)col * T::BN;
        t.w += (int64_t)expert * g.N * g.K;
        t.sw += (int64_t)expert * g.N;
    } else {
        const int band = tl / (g.group * g.tiles_n);
        const int in_band = tl - band * g.group * g.tiles_n;
        const int band_rows = min(g.group, g.tiles_m - band * g.group);
        t.m0 = (int64_t)(band * g.group + in_band % band_rows) * T::BM;
        t.n0 = (int64_t)(in_band / band_rows) * T::BN;
        t.m1 = g.M;
    }
    return true;
}

// This wave's copies global -> LDS. Instruction t moves 8 rows of A (t < A_INSTR), then of W;
// lane L fills LDS row L / 8 of those, physical chunk L % 8. VARIANT makes the type unique to
// each kernel instantiation: the host pass emits a launch stub for only one kernel among those
// that share such a type.
template <class T, int VARIANT, int STREAM>
struct Int8Dma {
    rsrc_t ra, rw;
    uint32_t off[T::IPW];
    int wave, chunk_byte, K;

    // the first tile row of instruction t
    __device__ __forceinline__ int row_of(int t) const {
        return 8 * (T::NW * (t < T::A_INSTR ? t : t - T::A_INSTR) + wave);
    }

    __device__ __forceinline__ Int8Dma(const Int8Args &g, const TileAt &at, int wave_, int lane)
        : wave(wave_), K((int)g.K) {
        const int sub = lane >> 3;
        const int64_t mrows = at.m1 - at.m0 < T::BM ? at.m1 - at.m0 : T::BM;
        const int64_t nrows = g.N - at.n0 < T::BN ? g.N - at.n0 : T::BN;
        rw = make_rsrc(at.w + at.n0 * K, nrows * K);
        ra = g.rows ? make_rsrc(g.a, g.tokens * K) : make_rsrc(g.a + at.m0 * K, mrows * K);
        chunk_byte = swz_chunk(sub, lane & 7) << 4;   // (rows 8 i + sub: their swizzle is sub's)
#pragma unroll
        for (int t = 0; t < T::IPW; ++t) {
            const int row = row_of(t) + sub;
            if (t < T::A_INSTR && g.rows) {
                const int token = row < mrows ? g.rows[at.m0 + row] : -1;
                off[t] = token >= 0 && token < g.tokens ? (uint32_t)token * (uint32_t)K + chunk_byte : kNowhere;
            } else {
                off[t] = (uint32_t)(row * K) + chunk_byte;
            }
        }
    }

    // copies first .. first + count - 1 (constants where this is inlined) of K step ks into the
    // stage buffer at `base`. Bytes past K (and steps past the last) read as zero, so that what the other
    // operand holds there counts for nothing.
    __device__ __forceinline__ void issue(uint8_t *base, int ks, int first = 0, int count = T::IPW) const {
        const int koff = __builtin_amdgcn_readfirstlane(ks * KB);
        const bool past = koff + chunk_byte >= K;
#pragma unroll
        for (int t = 0; t < T::IPW; ++t) {
            if (t < first || t >= first + count) continue;
            const uint32_t at = past ? kNowhere : off[t];
            if (t < T::A_INSTR)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void *)(base + row_of(t) * KB), 16, at, koff, 0, 0);
            else
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void *)(base + T::A_BYTES + row_of(t) * KB), 16, at,
                                                         koff, 0, STREAM ? kNonTemporal : 0);
        }
    }
};

template <class T, int OUT_BF16>
struct Int8Epilogue {
    static constexpr int OB = OUT_BF16 ? 2 : 4, EPC = 16 / OB;
    static constexpr int ROW_WORDS = T::BN * OB / 4, TARGET = OUT_BF16 ? 8 : 16;
    static constexpr int LDS_ROW = 4 * (ROW_WORDS + ((TARGET - ROW_WORDS) % 64 + 64) % 64);
    static constexpr int RG = T::WAVES_M * 16, CPR = T::BN * OB / 16;
    static constexpr int STAGES = T::STAGE * T::NSTAGE;
    static constexpr int IPR0 = STAGES / (RG * LDS_ROW), IPR = IPR0 < T::SUB_M ? IPR0 : T::SUB_M;
    static_assert(IPR >= 1, "epilogue staging does not fit");
};

// The accumulators' scaled rows go through LDS and leave in whole 128-byte pieces, masked to
// the tile's rows and to N. (Stored straight from the fragments each line would be written in
// 8-byte pieces by several instructions.) Begins with a workgroup barrier.
//
// The large tiles' outputs bypass the caches, which hold what the other tiles read, where the rows
// are whole 64-byte blocks: 16384 x 7168 x 7168 619 -> 601 us, x 128 86 -> 77. (With rows of other
// lengths the blocks that two stores share cost more: 8903 x 4080 x 256 37 -> 43. Small outputs
// are read again soon: 64 x 7168 x 2048 and a reader of it 9.6 -> 10.1.)
template <class T, int OUT_BF16>
__device__ __forceinline__ void store_tile(const Int8Args &g, const TileAt &at, uint8_t *smem, int lane, int wm, int wn,
                                           const i32x4 (&acc)[T::SUB_M][T::SUB_N]) {
    using E = Int8Epilogue<T, OUT_BF16>;
    constexpr int OB = E::OB, EPC = E::EPC, LDS_ROW = E::LDS_ROW, RG = E::RG, IPR = E::IPR, CPR = E::CPR;
    constexpr int SUB_M = T::SUB_M, SUB_N = T::SUB_N, WN = T::WN;
    const int frow = lane & 15, kg = lane >> 4;
    const bool whole = T::NW == 8 && g.N * OB % 64 == 0 && reinterpret_cast<uintptr_t>(g.y) % 64 == 0;
    f32x4 scale_n[SUB_N], bias[SUB_N];
#pragma unroll
    for (int j = 0; j < SUB_N; ++j) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int64_t n = at.n0 + wn * WN + 16 * j + 4 * kg + r;
            scale_n[j][r] = n < g.N && g.K > 0 ? at.sw[n] : 0.0f;
            bias[j][r] = g.bias && n < g.N ? g.bias[n] : 0.0f;
        }
    }
    float scale_m[SUB_M];
#pragma unroll
    for (int i = 0; i < SUB_M; ++i) {
        int64_t m = at.m0 + T::row(wm, i) + frow;
        scale_m[i] = 0.0f;
        if (m < at.m1 && g.K > 0) {   // (with K = 0 there may be no scales)
            if (g.rows) m = g.rows[m];
            if (m >= 0 && m < g.tokens) scale_m[i] = g.sa[m];
        }
    }
#pragma unroll
    for (int i0 = 0; i0 < SUB_M; i0 += IPR) {
        __syncthreads();
#pragma unroll
        for (int ii = 0; ii < IPR; ++ii) {
            if (i0 + ii < SUB_M) {
                uint8_t *rowp = smem + (ii * RG + wm * 16 + frow) * LDS_ROW;
#pragma unroll
                for (int j = 0; j < SUB_N; ++j) {
                    const int col = wn * WN + 16 * j + 4 * kg;
                    f32x4 v;
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        v[r] = (float)acc[i0 + ii][j][r] * scale_m[i0 + ii] * scale_n[j][r] + bias[j][r];
                    if constexpr (OUT_BF16)
                        *reinterpret_cast<u32x2 *>(rowp + col * 2) =
                            u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
                    else
                        *reinterpret_cast<f32x4 *>(rowp + col * 4) = v;
                }
            }
        }
        __syncthreads();
        const int groups = (SUB_M - i0) < IPR ? (SUB_M - i0) : IPR;
        const int chunks = groups * RG * CPR;
        // (a loop for either policy: two stores in one loop's branches would be merged into a plain one)
        auto copy_out = [&](auto stream) {
            for (int c = threadIdx.x; c < chunks; c += T::NW * 64) {
                const int r = c / CPR, cb = c - r * CPR;
                const int ii = r / RG, within = r - ii * RG;
                const int64_t m = at.m0 + T::row(within >> 4, i0 + ii) + (within & 15);
                const int64_t n = at.n0 + cb * EPC;
                if (m >= at.m1 || n >= g.N) continue;
                const uint8_t *src = smem + r * LDS_ROW + cb * 16;
                uint8_t *yp = reinterpret_cast<uint8_t *>(g.y) + (m * g.N + n) * OB;
                if constexpr (decltype(stream)::value) {   // (N is a multiple of EPC)
                    __builtin_nontemporal_store(*reinterpret_cast<const u32x4 *>(src), reinterpret_cast<u32x4 *>(yp));
                } else if (n + EPC <= g.N) {
                    *reinterpret_cast<u32x4_any *>(yp) = *reinterpret_cast<const u32x4 *>(src);
                } else {
                    for (int e = 0; e < EPC && n + e < g.N; ++e) {
                        if constexpr (OUT_BF16)
                            reinterpret_cast<uint16_t *>(yp)[e] = reinterpret_cast<const uint16_t *>(src)[e];
                        else
                            reinterpret_cast<float *>(yp)[e] = reinterpret_cast<const float *>(src)[e];
                    }
                }
            }
        };
        if (whole) copy_out(std::true_type{});
        else copy_out(std::false_type{});
    }
}

__device__ __forceinline__ void wait_lgkm0() { __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (0 << 8) | (3 << 14)); }

// Tiles of 8 waves, two to a SIMD, that take turns: waves 0-3 and 4-7 are one barrier apart, so
// that in each interval between two barriers ("slot") one wave of a SIMD multiplies from
// registers while the other fills its own from LDS and queues copies. A wave's K step of 128
// bytes is PH phases (2 for BM = 256, 1 for 128), each a load slot and a multiply slot of 32
// MFMAs (512 cycles): phase 0 loads the step's W fragments and the wave's first 64 rows of A,
// phase 1 the other 64 rows, over the same registers. In a tile that is not FULL of rows, groups of
// 16 rows past the last are not multiplied (the branches cost a full tile 5%).
//
// Copies. A region of a stage buffer is free once both groups have loaded it, which each load
// slot ends by waiting for (lgkmcnt). With two phases and two stages, the copies of step ks + 2
// for W and the tile's first 128 rows are queued in load slot 1 of step ks, those of its other
// rows in load slot 0 of step ks + 1; with one phase and three stages, those of step ks + 2 in
// the load slot of step ks. Copies retire in order, and the count left open at the end of each
// load slot (IPW) covers exactly what the load slots before the data's use have queued since;
// the barrier then makes it visible. Steps past the last copy zeros, which keeps the counts
// the same.
//
// What bounds it: 16384 x 7168 x 7168 takes 500 us on zeros (3.4 POP/s: the matrix unit busy 0.78 of
// the cycles) and 600 us on normal data (2.8 POP/s), at a lower clock (about 1.6 GHz): the power limit. The
// 32x32x32 instruction, at half the K and so twice the accumulator traffic, has fewer cycles
// and yet takes 685 us.
template <class T, int FULL, int VARIANT, int STREAM, int OUT_BF16>
__device__ __forceinline__ void turns(const Int8Args &g, const TileAt &at, uint8_t *smem) {
    constexpr int SUB_M = T::SUB_M, SUB_N = T::SUB_N, PH = SUB_M / 4;
    static_assert(PH == 1 || PH == 2, "phases");
    constexpr int I0 = T::A_INSTR / 2;   // two phases: copies of the first 128 rows
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave >> 2, wn = wave & 3;
    const int nks = (int)((g.K + KB - 1) / KB);
    const Int8Dma<T, VARIANT, STREAM> dma(g, at, wave, lane);
    const int rows = (int)(at.m1 - at.m0 < T::BM ? at.m1 - at.m0 : T::BM);

    i32x4 acc[SUB_M][SUB_N];
#pragma unroll
    for (int i = 0; i < SUB_M; ++i)
#pragma unroll
        for (int j = 0; j < SUB_N; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    const int frow = lane & 15, kg = lane >> 4;
    const int lo = frow * KB + (swz_chunk(frow, kg) << 4);
    const int hi = frow * KB + (swz_chunk(frow, 4 + kg) << 4);
    const int w_base = T::A_BYTES + wn * T::WN * KB;

    if constexpr (PH == 2) {
        dma.issue(smem, 0, T::A_INSTR, T::W_INSTR);
        dma.issue(smem, 0, 0, I0);
        dma.issue(smem, 0, I0, I0);
        dma.issue(smem + T::STAGE, 1, T::A_INSTR, T::W_INSTR);
        dma.issue(smem + T::STAGE, 1, 0, I0);
    } else {
        dma.issue(smem, 0);
        dma.issue(smem + T::STAGE, 1);
    }
    wait_vmcnt<T::IPW>();
    lds_barrier();
    if (wave >= 4) lds_barrier();   // one slot behind

    uint8_t *stage = smem, *stage1 = smem + T::STAGE;   // of steps ks and ks + 1
    for (int ks = 0; ks < nks; ++ks) {
        uint8_t *stage2 = stage1 + T::STAGE == smem + T::STAGE * T::NSTAGE ? smem : stage1 + T::STAGE;
        u32x4 wf[SUB_N][2];
#pragma unroll
        for (int ph = 0; ph < PH; ++ph) {
            u32x4 xf[4][2];
            if (ph == 0) {
#pragma unroll
                for (int j = 0; j < SUB_N; ++j) {
                    wf[j][0] = *reinterpret_cast<const u32x4 *>(stage + w_base + 16 * j * KB + lo);
                    wf[j][1] = *reinterpret_cast<const u32x4 *>(stage + w_base + 16 * j * KB + hi);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                xf[i][0] = *reinterpret_cast<const u32x4 *>(stage + T::row(wm, 4 * ph + i) * KB + lo);
                xf[i][1] = *reinterpret_cast<const u32x4 *>(stage + T::row(wm, 4 * ph + i) * KB + hi);
            }
            if constexpr (PH == 1) {
                dma.issue(stage2, ks + 2);
            } else if (ph == 0) {
                dma.issue(stage1, ks + 1, I0, I0);
            } else {
                dma.issue(stage2, ks + 2, T::A_INSTR, T::W_INSTR);
                dma.issue(stage2, ks + 2, 0, I0);
            }
            __builtin_amdgcn_sched_barrier(0);   // the waits stay behind the loads and copies
            wait_lgkm0();
            wait_vmcnt<T::IPW>();
            lds_barrier();
            __builtin_amdgcn_s_setprio(1);
            if constexpr (FULL) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < SUB_N; ++j)
                            acc[4 * ph + i][j] = mfma_i8(wf[j][h], xf[i][h], acc[4 * ph + i][j]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (T::row(wm, 4 * ph + i) < rows) {
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int j = 0; j < SUB_N; ++j)
                                acc[4 * ph + i][j] = mfma_i8(wf[j][h], xf[i][h], acc[4 * ph + i][j]);
                    }
                }
            }
            __builtin_amdgcn_s_setprio(0);
            __builtin_amdgcn_sched_barrier(0);
            lds_barrier();
        }
        stage = stage1;
        stage1 = stage2;
    }
    if (wave < 4) lds_barrier();
    wait_vmcnt<0>();   // the copies past the last step, before LDS takes the output
    store_tile<T, OUT_BF16>(g, at, smem, lane, wm, wn, acc);
}

// Tiles of BM x 256. With BM = 256 a tile with at most 128 rows (an expert's last, or only one)
// takes half the phases.
template <int BM, int OUT_BF16, int GROUPED>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void int8_turns_kernel(Int8Args g) {
    using T2 = Int8Tile<256, 256, 8, 2, 2>;
    using T1 = Int8Tile<128, 256, 8, 2, 3>;
    constexpr int A = T2::STAGE * T2::NSTAGE, B = T1::STAGE * T1::NSTAGE, VARIANT = OUT_BF16 * 2 + GROUPED;
    __shared__ __attribute__((aligned(16))) uint8_t smem[A > B ? A : B];
    TileAt at;
    if constexpr (BM == 256) {
        if (!find_tile<T2, GROUPED>(g, at)) return;
        const int64_t rows = at.m1 - at.m0;
        if (rows >= 256) {
            turns<T2, 1, VARIANT, 0, OUT_BF16>(g, at, smem);
        } else if (GROUPED && at.stream) {
            if (rows > 128) turns<T2, 0, VARIANT, GROUPED, OUT_BF16>(g, at, smem);
            else turns<T1, 0, VARIANT, GROUPED, OUT_BF16>(g, at, smem);
        } else {
            if (rows > 128) turns<T2, 0, VARIANT, 0, OUT_BF16>(g, at, smem);
            else turns<T1, 0, VARIANT, 0, OUT_BF16>(g, at, smem);
        }
    } else {
        if (!find_tile<T1, GROUPED>(g, at)) return;
        if (at.m1 - at.m0 >= 128) turns<T1, 1, 8 + VARIANT, 0, OUT_BF16>(g, at, smem);
        else if (GROUPED && at.stream) turns<T1, 0, 8 + VARIANT, GROUPED, OUT_BF16>(g, at, smem);
        else turns<T1, 0, 8 + VARIANT, 0, OUT_BF16>(g, at, smem);
    }
}

// One or two rows of up to 8192 elements, as bf16 (a decoded token): 32 channels a workgroup. W comes
// through LDS, in stages of four times 128 bytes of K, while the rows are quantised into LDS by every
// workgroup for itself. Waves 0 and 1 take 16 channels each and the first half of every 128 bytes,
// waves 2 and 3 the other half. Bound by the read of W: 1 x 7168 x 7168 9.8 us, of which its 51 MB
// are 9 at 5.7 TB/s (with W straight into registers, half a line of a row at a time, 12.1). Three stages,
// so that two workgroups share a CU: with four 1 x 10240 x 7168 takes 17.2 instead of 13.4.
constexpr int kRowRows = 2, kRowK = 8192, kRowN = 32;
template <int OUT_BF16>
__global__ __launch_bounds__(256) void int8_row_kernel(Int8FewArgs g) {
    constexpr int BN = kRowN, SUBS = 4, STAGES = 3, STEP = BN * KB, STAGE = SUBS * STEP, PITCH = kRowK + 16;
    __shared__ __attribute__((aligned(16))) uint8_t ring[STAGES * STAGE];
    __shared__ __attribute__((aligned(16))) uint8_t codes[kRowRows * PITCH];
    __shared__ uint32_t tops[4][kRowRows];
    __shared__ i32x4 part[2][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row = lane & 15, kg = lane >> 4, K = g.K, M = g.M;
    const int64_t n0 = (int64_t)blockIdx.x * BN;
    const int nw = (int)(g.N - n0 < BN ? g.N - n0 : BN);
    const rsrc_t rw = make_rsrc(g.w + n0 * K, (int64_t)nw * K), rx = make_rsrc(g.x, (int64_t)M * K * 2);

    constexpr int NV = kRowK / 8 / 256;   // pieces of 8 elements a thread keeps of a row
    u32x4 v[kRowRows][NV];
    // the rows first: loads return in order, and these are needed before W
#pragma unroll
    for (int m = 0; m < kRowRows; ++m) {
        if (m < M) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int p = threadIdx.x + 256 * i;
                v[m][i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                        rx, 8 * p < K ? (uint32_t)(2 * (m * K + 8 * p)) : kNowhere, 0, 0));
            }
        }
    }
    __builtin_amdgcn_sched_barrier(0);
    // Copies of a stage: each wave 8 rows of W, lane L the physical chunk L % 8 of row L / 8; bytes past K,
    // and channels past N, read as zero, which makes what `codes` holds there count for nothing
    const int chunk_byte = swz_chunk(lane >> 3, lane & 7) << 4;
    const uint32_t off = (uint32_t)((8 * wave + (lane >> 3)) * K) + chunk_byte;
    auto copy = [&](uint8_t *stage, int ks) {
#pragma unroll
        for (int s = 0; s < SUBS; ++s) {
            const int koff = __builtin_amdgcn_readfirstlane((ks * SUBS + s) * KB);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void *)(stage + s * STEP + 8 * wave * KB), 16,
                                                     koff + chunk_byte >= K ? kNowhere : off, koff, 0, 0);
        }
    };
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) copy(ring + s * STAGE, s);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int m = 0; m < kRowRows; ++m) {
        if (m < M) {
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const uint32_t b = absmax_bits8(v[m][i]);
                top = top > b ? top : b;
            }
            top = wave_umax(top);
            if (lane == 0) tops[wave][m] = top;
        }
    }
    wait_lgkm0();   // (a barrier that waits for LDS, not for the copies)
    lds_barrier();
    float scale = 0.0f;   // of this lane's row
#pragma unroll
    for (int m = 0; m < kRowRows; ++m) {
        if (m < M) {
            uint32_t top = tops[0][m];
#pragma unroll
            for (int w = 1; w < 4; ++w) top = top > tops[w][m] ? top : tops[w][m];
            const RowScale r = row_scale(top);
            scale = row == m ? r.s : scale;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int p = threadIdx.x + 256 * i;
                if (8 * p < K) *reinterpret_cast<u32x2 *>(codes + m * PITCH + 8 * p) = codes8(v[m][i], r);
            }
        }
    }

    const int cg = wave & 1, half = wave >> 1;
    const int w_at = (16 * cg + row) * KB + (swz_chunk(row, 4 * half + kg) << 4);
    const uint8_t *x_at = codes + (row < M ? row : 0) * PITCH + 64 * half + 16 * kg;
    i32x4 acc = {0, 0, 0, 0};
    const int nks = (K + SUBS * KB - 1) / (SUBS * KB);
    uint8_t *stage = ring, *last = ring + (STAGES - 1) * STAGE;   // `last`: of the step before
    for (int ks = 0; ks < nks; ++ks) {
        __builtin_amdgcn_sched_barrier(0);
        wait_lgkm0();                                // (the codes, and the step before's reads)
        wait_vmcnt<SUBS *(STAGES - 2)>();            // this step has landed
        lds_barrier();
        copy(last, ks + STAGES - 1);
#pragma unroll
        for (int s = 0; s < SUBS; ++s) {
            const u32x4 w = *reinterpret_cast<const u32x4 *>(stage + s * STEP + w_at);
            u32x4 x = {0, 0, 0, 0};
            if (row < M) x = *reinterpret_cast<const u32x4 *>(x_at + (ks * SUBS + s) * KB);
            acc = mfma_i8(w, x, acc);
        }
        last = stage;
        stage = stage + STAGE == ring + STAGES * STAGE ? ring : stage + STAGE;
    }
    wait_vmcnt<0>();
    if (half == 1) part[cg][lane] = acc;
    __syncthreads();
    const int64_t n = n0 + 16 * cg + 4 * kg;
    if (half == 1 || row >= M || n >= g.N) return;
    const i32x4 sum = acc + part[cg][lane];
    f32x4 out;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int64_t nr = n + r < g.N ? n + r : g.N - 1;
        out[r] = (float)sum[r] * scale * (K > 0 ? g.sw[nr] : 0.0f) + (g.bias ? g.bias[nr] : 0.0f);
    }
    store4<OUT_BF16>(g.y, row * g.N + n, out, g.N - n);
}

// Smaller tiles of 4 waves, for shapes with too few of the large ones. Their time is K's steps one
// after another, each waiting for memory, so as many stages as fit are in flight (128 KB or more a
// CU: 64 experts' 4096 x 7168 at 1.5 rows, 32 x 128, 158 us, W read at 7.0 TB/s; 64 x 7168 x 7168 11.2 us).
// Two register sets hold the fragments of two steps: the MFMAs of step ks take one while the
// other is filled with step ks + 1. A stage buffer is free once its step is in registers
// everywhere (lgkmcnt, then the barrier), and takes the copies of step ks + NSTAGE; steps past
// the last copy zeros, so that the count left open always covers NSTAGE - 1 steps.
template <class T>
__device__ __forceinline__ u32x4 read_piece(const uint8_t *stage, int f, int wm, int w_base, int at) {
    return *reinterpret_cast<const u32x4 *>(
        stage + (f < T::SUB_N ? w_base + 16 * f * KB : T::row(wm, f - T::SUB_N) * KB) + at);
}

// A wave issues in order, and a copy waits for the CU's one address unit (16 cycles a copy): queued
// in a row ahead of the MFMAs, the copies and LDS reads add to their time instead of hiding
// behind it. So each row group's MFMAs are preceded by their share of both. A step is S times 128
// bytes of K: with the smallest tile the barrier and the LDS latency of a step take longer than
// its copies, so it is made of two (64 x 576 x 7168 8.8 -> 7.3 us; 32 x 64 tiles gain nothing).
template <class T, int S, class Dma>
__device__ __forceinline__ void deep_step(int ks, const Dma &dma, uint8_t *stage, const uint8_t *stage1, int wm,
                                          int w_base, int lo, int hi,
                                          const u32x4 (&wf)[S][T::SUB_N][2], const u32x4 (&xf)[S][T::SUB_M][2],
                                          u32x4 (&wf_next)[S][T::SUB_N][2], u32x4 (&xf_next)[S][T::SUB_M][2],
                                          i32x4 (&acc)[T::SUB_M][T::SUB_N]) {
    constexpr int PER = 2 * T::SUB_M, GROUPS = PER * S, RPER = 2 * (T::SUB_M + T::SUB_N), READS = RPER * S;
    constexpr int COPIES = T::IPW * S, AHEAD = T::NSTAGE / S;
    __builtin_amdgcn_sched_barrier(0);          // the waits stay behind the previous step's MFMAs
    wait_lgkm0();                               // step ks is in registers
    wait_vmcnt<COPIES * (AHEAD - 2)>();         // step ks + 1 has landed
    lds_barrier();
#pragma unroll
    for (int q = 0; q < GROUPS; ++q) {
#pragma unroll
        for (int r = q * READS / GROUPS; r < (q + 1) * READS / GROUPS; ++r) {
            const int sub = r / RPER, f = r % RPER / 2;
            const u32x4 v = read_piece<T>(stage1 + sub * T::STAGE, f, wm, w_base, r & 1 ? hi : lo);
            if (f < T::SUB_N) wf_next[sub][f][r & 1] = v;
            else xf_next[sub][f - T::SUB_N][r & 1] = v;
        }
#pragma unroll
        for (int c = q * COPIES / GROUPS; c < (q + 1) * COPIES / GROUPS; ++c)
            dma.issue(stage + c / T::IPW * T::STAGE, (ks + AHEAD) * S + c / T::IPW, c % T::IPW, 1);
        const int sub = q / PER, h = q % PER / T::SUB_M, i = q % T::SUB_M;
#pragma unroll
        for (int j = 0; j < T::SUB_N; ++j) acc[i][j] = mfma_i8(wf[sub][j][h], xf[sub][i][h], acc[i][j]);
        __builtin_amdgcn_sched_barrier(0);
    }
}

template <class T, int S, int VARIANT, int STREAM, int OUT_BF16>
__device__ __forceinline__ void deep(const Int8Args &g, const TileAt &at, uint8_t *smem) {
    constexpr int SUB_M = T::SUB_M, SUB_N = T::SUB_N, NSTAGE = T::NSTAGE, RPER = 2 * (SUB_M + SUB_N);
    static_assert(NSTAGE % S == 0 && NSTAGE / S >= 3, "stages");
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave & 1, wn = wave >> 1;
    const int nks = (int)((g.K + KB * S - 1) / (KB * S));
    const Int8Dma<T, VARIANT, STREAM> dma(g, at, wave, lane);

    i32x4 acc[SUB_M][SUB_N];
#pragma unroll
    for (int i = 0; i < SUB_M; ++i)
#pragma unroll
        for (int j = 0; j < SUB_N; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    const int frow = lane & 15, kg = lane >> 4;
    const int lo = frow * KB + (swz_chunk(frow, kg) << 4);
    const int hi = frow * KB + (swz_chunk(frow, 4 + kg) << 4);
    const int w_base = T::A_BYTES + wn * T::WN * KB;

#pragma unroll
    for (int s = 0; s < NSTAGE; ++s) dma.issue(smem + s * T::STAGE, s);
    wait_vmcnt<T::IPW *(NSTAGE - S)>();
    lds_barrier();
    u32x4 wf0[S][SUB_N][2], xf0[S][SUB_M][2], wf1[S][SUB_N][2], xf1[S][SUB_M][2];
#pragma unroll
    for (int r = 0; r < RPER * S; ++r) {
        const int sub = r / RPER, f = r % RPER / 2;
        const u32x4 v = read_piece<T>(smem + sub * T::STAGE, f, wm, w_base, r & 1 ? hi : lo);
        if (f < SUB_N) wf0[sub][f][r & 1] = v;
        else xf0[sub][f - SUB_N][r & 1] = v;
    }
    uint8_t *const end = smem + NSTAGE * T::STAGE;
    uint8_t *stage = smem;
    for (int ks = 0; ks < nks; ks += 2) {
        // (with an odd number of steps the last one here multiplies zeros)
        uint8_t *stage1 = stage + S * T::STAGE == end ? smem : stage + S * T::STAGE;
        uint8_t *stage2 = stage1 + S * T::STAGE == end ? smem : stage1 + S * T::STAGE;
        deep_step<T, S>(ks, dma, stage, stage1, wm, w_base, lo, hi, wf0, xf0, wf1, xf1, acc);
        deep_step<T, S>(ks + 1, dma, stage1, stage2, wm, w_base, lo, hi, wf1, xf1, wf0, xf0, acc);
        stage = stage2;
    }
    wait_lgkm0();
    wait_vmcnt<0>();   // the copies past the last step, before LDS takes the output
    store_tile<T, OUT_BF16>(g, at, smem, lane, wm, wn, acc);
}

template <int BM, int BN, int NSTAGE, int OUT_BF16, int GROUPED>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 2))) void int8_deep_kernel(Int8Args g) {
    using T = Int8Tile<BM, BN, 4, 2, NSTAGE>;
    constexpr int VARIANT = 4 + OUT_BF16 * 2 + GROUPED;
    __shared__ __attribute__((aligned(16))) uint8_t smem[T::STAGE * NSTAGE];
    TileAt at;
    if (!find_tile<T, GROUPED>(g, at)) return;
    constexpr int S = BN == 32 ? 2 : 1;
    if (GROUPED && at.stream) deep<T, S, VARIANT, GROUPED, OUT_BF16>(g, at, smem);
    else deep<T, S, VARIANT, 0, OUT_BF16>(g, at, smem);
}

template <int U, int QUANT>
hipError_t launch_few(const Int8FewArgs &a, bool out_bf16, hipStream_t stream) {
    const int64_t units = (a.N + 15) / 16;
    if (units * 256 > 0xFFFFFFFFll) return hipErrorInvalidValue;
    const dim3 grid((unsigned)units), block(256);
    if (out_bf16) int8_few_kernel<U, QUANT, 1><<<grid, block, 0, stream>>>(a);
    else int8_few_kernel<U, QUANT, 0><<<grid, block, 0, stream>>>(a);
    return hipGetLastError();
}

// The launch's tiles: their counts (grouped: an upper bound, full row blocks and a last one for each
// expert that has rows), and the tile rows walked per tile column (an XCD's ~32 resident tiles
// form a compact block). False if the grid would be too large.
bool lay_out(Int8Args &a, int BM, int BN, int threads) {
    a.tiles_m = (int)(a.offsets ? a.M / BM + (a.experts < a.M ? a.experts : a.M) : (a.M + BM - 1) / BM);
    a.tiles_n = (int)((a.N + BN - 1) / BN);
    int64_t best = -1;
    for (int gsz = 1; gsz <= 32; gsz *= 2) {
        const int64_t gg = gsz < a.tiles_m ? gsz : a.tiles_m, cols = (32 + gg - 1) / gg;
        const int64_t rows = gg * BM + (cols < a.tiles_n ? cols : a.tiles_n) * BN;
        if (best < 0 || rows < best) {
            best = rows;
            a.group = gsz;
        }
    }
    return (int64_t)a.tiles_m * a.tiles_n * threads <= 0xFFFFFFFFll;
}

template <int BM, int GROUPED>
hipError_t launch_turns(Int8Args a, bool out_bf16, hipStream_t stream) {
    if (!lay_out(a, BM, 256, 512)) return hipErrorInvalidValue;
    const dim3 grid((unsigned)(a.tiles_m * a.tiles_n)), block(512);
    if (out_bf16) int8_turns_kernel<BM, 1, GROUPED><<<grid, block, 0, stream>>>(a);
    else int8_turns_kernel<BM, 0, GROUPED><<<grid, block, 0, stream>>>(a);
    return hipGetLastError();
}

template <int BM, int BN, int NSTAGE, int GROUPED>
hipError_t launch_deep(Int8Args a, bool out_bf16, hipStream_t stream) {
    if (!lay_out(a, BM, BN, 256)) return hipErrorInvalidValue;
    const dim3 grid((unsigned)(a.tiles_m * a.tiles_n)), block(256);
    if (out_bf16) int8_deep_kernel<BM, BN, NSTAGE, 1, GROUPED><<<grid, block, 0, stream>>>(a);
    else int8_deep_kernel<BM, BN, NSTAGE, 0, GROUPED><<<grid, block, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_int8_quant(const uint16_t *x, int8_t *q, float *s, int64_t M, int64_t K, hipStream_t stream) {
    // Waves of a row, us: 16 x 2048 one 2.8, four 2.2, 2048 x 2048 3.7 / 5.0; 16 x 7168 four 3.0, sixteen 3.0,
    // 2048 x 7168 8.4 / 15.2; 16 x 20000 5.4 / 3.1, 8192 x 20000 96 / 89.
    const dim3 block(256), large(1024), four((unsigned)((M + 3) / 4)), one((unsigned)M);
    if (K <= 512) row_quant_kernel<1, 1><<<four, block, 0, stream>>>(x, q, s, M, K);
    else if (K <= 2048 && M <= 512) row_quant_kernel<4, 1><<<one, block, 0, stream>>>(x, q, s, M, K);
    else if (K <= 2048) row_quant_kernel<1, 4><<<four, block, 0, stream>>>(x, q, s, M, K);
    else if (K <= 8192) row_quant_kernel<4, 4><<<one, block, 0, stream>>>(x, q, s, M, K);
    else {
        // A grid counts at most 2^32 - 1 threads (more are not refused: their number wraps), so 2^22 rows
        // and more of 1024 threads each are several launches
        constexpr int64_t kRows = 0xFFFFFFFFll / 1024;
        for (int64_t m = 0; m < M; m += kRows) {
            const int64_t n = M - m < kRows ? M - m : kRows;
            const dim3 grid((unsigned)n);
            if (K <= 32768) row_quant_kernel<16, 4><<<grid, large, 0, stream>>>(x + m * K, q + m * K, s + m, n, K);
            else row_quant_kernel<16, 0><<<grid, large, 0, stream>>>(x + m * K, q + m * K, s + m, n, K);
            if (hipError_t e = hipGetLastError()) return e;
        }
    }
    return hipGetLastError();
}

hipError_t launch_int8_gemm(const int8_t *a, const float *sa, const int8_t *w, const float *sw, const float *bias,
                            void *y, bool out_bf16, int64_t M, int64_t N, int64_t K, hipStream_t stream) {
    // Few rows: against the tiles, us, W from memory: 1 x 1536 x 7168 6.7 / 9.1, 4 rows 7.3 / 9.1, 16 rows 9.5 / 9.2;
    // 1 x 4096 x 7168 7.6 / 10.5; 1 x 7168 x 7168 (two workgroups on most CUs) 12.6 / 11.8.
    if (M <= kFewRows && N <= 4096)
        return launch_few<8, 0>({a, sa, nullptr, w, sw, bias, y, N, (int)M, (int)K}, out_bf16, stream);
    const Int8Args g{a, sa, w, sw, bias, y, nullptr, nullptr, M, N, K, M, 0, 0, 0, 1, false};
    // The tile by its time: rounds of 256 tiles (one a CU), each an epilogue and K's steps. The
    // constants are fitted to times at K = 512 and 7168, N = 1536 and 7168, M = 16 to 4096 (us): the
    // first round's step, a later round's (less where two workgroups share a CU's waits), the epilogue.
    const double steps = (double)((K + KB - 1) / KB);
    // (Tiles whose grid would pass 2^32 - 1 threads are left out: 2^30 rows have too many of 64.)
    auto time = [&](int bm, int bn, double first, double more, double end, int threads = 256) {
        const int64_t tiles = ((M + bm - 1) / bm) * ((N + bn - 1) / bn);
        if (tiles * threads > 0xFFFFFFFFll) return HUGE_VAL;
        const double rounds = (double)((tiles + 255) / 256);
        return steps * (first + more * (rounds - 1.0)) + end * rounds;
    };
    const double t[7] = {time(32, 32, 0.105, 0.085, 1.0), time(32, 64, 0.155, 0.125, 1.1),
                         time(64, 64, 0.21, 0.18, 1.4),   time(64, 128, 0.34, 0.27, 1.5),
                         time(128, 128, 0.45, 0.53, 5.0), time(128, 256, 0.75, 0.83, 5.7, 512),
                         time(256, 256, 1.3, 1.5, 8.0, 512)};
    int best = 0;
    for (int i = 1; i < 7; ++i)
        if (t[i] < t[best]) best = i;
    if (t[best] == HUGE_VAL) return hipErrorInvalidValue;
    switch (best) {
    case 0: return launch_deep<32, 32, 8, 0>(g, out_bf16, stream);
    case 1: return launch_deep<32, 64, 6, 0>(g, out_bf16, stream);
    case 2: return launch_deep<64, 64, 5, 0>(g, out_bf16, stream);
    case 3: return launch_deep<64, 128, 3, 0>(g, out_bf16, stream);
    case 4: return launch_deep<128, 128, 4, 0>(g, out_bf16, stream);
    case 5: return launch_turns<128, 0>(g, out_bf16, stream);
    default: return launch_turns<256, 0>(g, out_bf16, stream);
    }
}

// Whether a linear layer is one launch, and by which kernel (1: int8_row_kernel, 2: int8_few_kernel). One
// launch against two, us: 2, 8 x 4096 x 2048 5.6 / 7.0, 16 rows 8.3 / 7.3, 8 x 32768 x 2048 17 / 16 (the rows are
// quantised over and over); 1, 1 x 512 x 2560 4.4 / 6.1, 1 x 7168 x 7168 10.0 / 13.1, 2 x 32768 x 7168 42.8 / 44.7.
// (A grid counts at most 2^32 - 1 threads.)
constexpr int64_t kRowMaxN = 0xFFFFFFFFll / 256 * kRowN;
static int one_launch(int64_t M, int64_t N, int64_t K) {
    if (M <= kFewRows && K <= kFewQuantK && N <= 16384) return 2;
    if (M <= kRowRows && K <= kRowK && N <= kRowMaxN) return 1;
    return 0;
}

// Quantised rows of a linear layer between the two launches: the codes, then the scales
size_t int8_linear_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    return one_launch(M, N, K) ? 0 : (size_t)(M * K + 4 * M);
}

hipError_t launch_int8_linear(const uint16_t *x, const int8_t *w, const float *sw, const float *bias, void *y,
                              bool out_bf16, int64_t M, int64_t N, int64_t K, void *workspace, hipStream_t stream) {
    const Int8FewArgs few{nullptr, nullptr, x, w, sw, bias, y, N, (int)M, (int)K};
    switch (one_launch(M, N, K)) {
    case 1: {
        const dim3 grid((unsigned)((N + kRowN - 1) / kRowN)), block(256);
        if (out_bf16) int8_row_kernel<1><<<grid, block, 0, stream>>>(few);
        else int8_row_kernel<0><<<grid, block, 0, stream>>>(few);
        return hipGetLastError();
    }
    case 2: return launch_few<4, 1>(few, out_bf16, stream);
    }
    int8_t *q = static_cast<int8_t *>(workspace);
    float *s = reinterpret_cast<float *>(q + M * K);
    if (hipError_t e = launch_int8_quant(x, q, s, M, K, stream)) return e;
    return launch_int8_gemm(q, s, w, sw, bias, y, out_bf16, M, N, K, stream);
}

hipError_t launch_int8_grouped_gemm(const int8_t *a, const float *sa, const int8_t *w, const float *sw,
                                    const int64_t *offsets, const int32_t *rows, void *y, bool out_bf16,
                                    int64_t experts, int64_t M, int64_t tokens, int64_t N, int64_t K,
                                    hipStream_t stream) {
    const Int8Args g{a, sa, w, sw, nullptr, y, offsets, rows, M, N, K, tokens, (int)experts, 0, 0, 1,
                     experts * N * K > kLastLevelCache};
    // By the average rows of an expert (its true count is on the device). Measured in us at 1.5 / 15 /
    // 24 / 48 / 96 / 192 rows of each of 64 experts:
    //     4096 x 7168   32 x 128 158 / 280 / 326 / 432 / 606 / 976    64 x 128 165 / 287 / 296 / 365 / 482 / 689
    //                  128 x 256 189 / 286 / 303 / 357 / 407 / 562   256 x 256 190 / 286 / 304 / 336 / 389 / 500
    //      512 x 1024 at 30 / 96 / 192  10 / 17 / 28,  11 / 17 / 22,  13 / 15 / 27,  13 / 22 / 25
    // With few tiles the smallest that still all run at once (a CU reads some 65 GB/s from memory, so the
    // more of them the better): 12 experts' 412 x 4752 at 16 rows 32 x 32 11, 32 x 64 17, 64 x 64 17; 29 experts'
    // 169 x 4912 at 38 rows 32 x 64 12, 64 x 64 15, 64 x 128 21; 53 experts' 106 x 3328 at 72 rows 11, 10, 13; 48 experts' 300 x 4000 at
    // 52 rows 64 x 128 19, 128 x 256 34. Between the last two by rounds of 256 tiles where they are few,
    // blocks of 256 rows taking 1.5 times as long (few are full): 32 experts' 1408 x 2048 at 250 rows 42
    // against 59; 8 experts' 4096 x 7168 at 128 rows 48 / 79, at 256 92 / 81. With many rounds the larger
    // blocks, which read W less often (64 experts of 144 rows each 468 / 372).
    const int64_t mean = M / experts;
    auto tiles = [&](int bm, int bn) {   // an expert's last row block counted as half
        return (M / bm + (experts < M ? experts : M) / 2) * ((N + bn - 1) / bn);
    };
    if (tiles(32, 32) <= 256) return launch_deep<32, 32, 8, 1>(g, out_bf16, stream);
    if (tiles(32, 64) <= 256) return launch_deep<32, 64, 6, 1>(g, out_bf16, stream);
    if (mean < 16) return launch_deep<32, 128, 4, 1>(g, out_bf16, stream);
    if (tiles(64, 64) <= 256) return launch_deep<64, 64, 5, 1>(g, out_bf16, stream);
    if (mean < 32 || tiles(64, 128) <= 512) return launch_deep<64, 128, 3, 1>(g, out_bf16, stream);
    const int64_t rounds128 = (tiles(128, 256) + 255) / 256, rounds256 = (tiles(256, 256) + 255) / 256;
    if (rounds128 <= 2 && 2 * rounds128 <= 3 * rounds256) return launch_turns<128, 1>(g, out_bf16, stream);
    return launch_turns<256, 1>(g, out_bf16, stream);
}

}  // namespace fp8q
