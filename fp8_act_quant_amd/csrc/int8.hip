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

// 8 codes of 8 bf16 values over the row's scale
__device__ __forceinline__ u32x2 codes8(u32x4 v, float d) {
    u32x2 out;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t word = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const uint32_t u = v[2 * h + b / 2];
            const float x = b & 1 ? bf16hi_to_f32(u) : bf16lo_to_f32(u);
            const float q = __builtin_amdgcn_fmed3f(__builtin_rintf(x / d), -127.0f, 127.0f);
            word |= ((uint32_t)(int)q & 0xFFu) << (8 * b);
        }
        out[h] = word;
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

// WAVES waves to a row, which they keep in registers between the maximum and the codes where
// it has at most 512 * WAVES * NV elements (NV > 0), and read a second time where it is longer.
template <int WAVES, int NV>
__global__ __launch_bounds__(256) void row_quant_kernel(const uint16_t *x, int8_t *q, float *s, int64_t M, int64_t K) {
    constexpr int ROWS = 4 / WAVES, NT = 64 * WAVES, KEEP = NV > 0 ? NV : 1;
    __shared__ uint32_t part[4];
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
    const float scale = __uint_as_float(top << 16) * (1.0f / 127.0f);
    const float d = top ? scale : 1.0f;
    u32x2 *dst = reinterpret_cast<u32x2 *>(q + (in ? m : 0) * K);
    if constexpr (NV > 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (tid + i * NT < n) dst[tid + i * NT] = codes8(v[i], d);
    } else {
        for (int64_t i = tid; i < n; i += NT) dst[i] = codes8(src[i], d);
    }
    if (in && tid == 0) s[m] = scale;
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
};

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

// The expert and the block of `bm` of its rows that row block `unit` (of all experts' blocks,
// in order) is. Each wave finds it by itself, 64 experts at a time. False: there is no such block.
// Also gives the number of blocks of that expert before it.
__device__ __forceinline__ bool find_block(const Int8Args &g, int bm, int unit, int &expert, int64_t &row0,
                                           int64_t &row1) {
    const int lane = threadIdx.x & 63;
    int before = 0;
    for (int e0 = 0; e0 < g.experts; e0 += 64) {
        const int e = e0 + lane;
        int64_t r0 = 0, r1 = 0;
        if (e < g.experts) expert_rows(g, e, r0, r1);
        const int n = (int)((r1 - r0 + bm - 1) / bm);
        int sum = n;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(sum, d, 64);
            sum += lane >= d ? o : 0;
        }
        const int first = before + sum - n;
        const uint64_t hit = __ballot(unit >= first && unit < first + n);
        if (hit) {
            const int at = __builtin_ctzll(hit);
            expert = e0 + at;
            expert_rows(g, expert, r0, r1);
            row0 = r0 + (int64_t)(unit - __builtin_amdgcn_readlane(first, at)) * bm;
            row1 = r1;
            return true;
        }
        before += __builtin_amdgcn_readlane(sum, 63);
    }
    return false;
}

template <int OUT_BF16>
__device__ __forceinline__ void store4(void *y, int64_t at, const f32x4 &v, int64_t left, bool vec) {
    if constexpr (OUT_BF16) {
        uint16_t *p = reinterpret_cast<uint16_t *>(y) + at;
        const u32x2 u = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        if (vec && left >= 4) {
            *reinterpret_cast<u32x2 *>(p) = u;
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (r < left) p[r] = (uint16_t)(u[r / 2] >> (16 * (r & 1)));
        }
    } else {
        float *p = reinterpret_cast<float *>(y) + at;
        if (vec && left >= 4) {
            *reinterpret_cast<f32x4 *>(p) = v;
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (r < left) p[r] = v[r];
        }
    }
}

// Few rows (a decode step): every byte of W is read once and met by at most 16 * MT tokens, so
// the read of W is what counts. A workgroup takes 16 channels; its 4 waves take a quarter of K
// each, straight from memory into MFMA operands (no LDS: nothing is read twice), U steps of 64
// bytes a batch, the next batch in flight while this one is multiplied. The quarters are added
// in LDS, exactly.
template <int MT, int U, int OUT_BF16, int GROUPED>
__global__ __launch_bounds__(256) void int8_few_kernel(Int8Args g) {
    __shared__ i32x4 part[4][MT][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row = lane & 15, kg = lane >> 4;
    const int block = blockIdx.x / g.tiles_n;
    const int64_t n0 = (int64_t)(blockIdx.x - block * g.tiles_n) * 16;
    const int8_t *w = g.w;
    const float *sw = g.sw;
    int64_t m0, m1;
    if constexpr (GROUPED) {
        int expert;
        if (!find_block(g, 16 * MT, block, expert, m0, m1)) return;
        w += (int64_t)expert * g.N * g.K;
        sw += (int64_t)expert * g.N;
    } else {
        m0 = (int64_t)block * 16 * MT;
        m1 = g.M;
    }
    const int K = (int)g.K;
    const int nw = (int)(g.N - n0 < 16 ? g.N - n0 : 16);
    const rsrc_t rw = make_rsrc(w + n0 * K, (int64_t)nw * K);
    // (grouped: one buffer over all tokens; else over this block's)
    const int8_t *a0 = g.rows ? g.a : g.a + m0 * K;
    const rsrc_t ra = make_rsrc(a0, g.rows ? g.tokens * K : (m1 - m0 < 16 * MT ? m1 - m0 : 16 * MT) * K);
    uint32_t aoff[MT];
    int64_t token[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int64_t m = m0 + 16 * i + row;
        token[i] = -1;
        aoff[i] = kNowhere;
        if (m < m1) {
            token[i] = m;
            if (g.rows) {
                const int t = g.rows[m];
                token[i] = t >= 0 && t < g.tokens ? t : -1;
                if (token[i] >= 0) aoff[i] = (uint32_t)t * (uint32_t)K;
            } else {
                aoff[i] = (uint32_t)(16 * i + row) * (uint32_t)K;
            }
        }
    }
    const int steps = (K + 63) / 64;
    const int s0 = wave * steps / 4, s1 = (wave + 1) * steps / 4;

    i32x4 acc[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[i] = i32x4{0, 0, 0, 0};
    u32x4 wv[2][U], av[2][MT][U];
    auto load = [&](int b, int s) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = (s + u) * 64 + kg * 16;
            const bool in = s + u < s1 && k < K;
            const u32x4 z = {0, 0, 0, 0};
            wv[b][u] = z;
            if (s + u < s1)
                wv[b][u] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                         rw, in ? (uint32_t)(row * K + k) : kNowhere, 0, 0));
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                av[b][i][u] = z;
                if (s + u < s1)
                    av[b][i][u] = __builtin_bit_cast(
                        u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                   ra, in && aoff[i] != kNowhere ? aoff[i] + (uint32_t)k : kNowhere, 0, 0));
            }
        }
    };
    auto multiply = [&](int b) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < MT; ++i) acc[i] = mfma_i8(wv[b][u], av[b][i][u], acc[i]);
    };
    load(0, s0);
    for (int s = s0; s < s1; s += 2 * U) {
        load(1, s + U);
        multiply(0);
        load(0, s + 2 * U);
        multiply(1);
    }

#pragma unroll
    for (int i = 0; i < MT; ++i) part[wave][i][lane] = acc[i];
    __syncthreads();
    const bool vec = (g.N & 3) == 0 && (reinterpret_cast<uintptr_t>(g.y) & 15) == 0;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        if ((i & 3) != wave) continue;
        i32x4 sum = part[0][i][lane];
#pragma unroll
        for (int v = 1; v < 4; ++v) sum += part[v][i][lane];
        const int64_t m = m0 + 16 * i + row, n = n0 + 4 * kg;
        if (m >= m1 || n >= g.N) continue;
        const float sm = token[i] >= 0 ? g.sa[token[i]] : 0.0f;
        f32x4 v;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int64_t nr = n + r < g.N ? n + r : g.N - 1;
            v[r] = (float)sum[r] * sm * sw[nr] + (g.bias ? g.bias[nr] : 0.0f);
        }
        store4<OUT_BF16>(g.y, m * g.N + n, v, g.N - n, vec);
    }
}

// Many rows: tiles of BM x BN in LDS, 8 or 4 waves of (BM / WAVES_M) x 64.
template <int BM_, int BN_, int NW_, int WAVES_M_>
struct Int8Tile {
    static constexpr int BM = BM_, BN = BN_, NW = NW_, WAVES_M = WAVES_M_, WAVES_N = NW_ / WAVES_M_;
    static constexpr int NSTAGE = 2;
    static constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N;
    static constexpr int SUB_M = WM / 16, SUB_N = WN / 16;
    static constexpr int A_BYTES = BM * KB, W_BYTES = BN * KB, STAGE = A_BYTES + W_BYTES;
    static constexpr int A_INSTR = BM / (8 * NW), W_INSTR = BN / (8 * NW), IPW = A_INSTR + W_INSTR;
    static_assert(WAVES_M * WAVES_N == NW && BM % (8 * NW) == 0 && BN % (8 * NW) == 0, "tile shape");
    static_assert(STAGE * NSTAGE <= 160 * 1024 && IPW < 64, "LDS budget");
};

// This wave's copies global -> LDS. Instruction t moves tile rows 8 (NW t + wave) .. + 7 of A
// (t < A_INSTR), then of W; lane L fills LDS row L / 8 of those, physical chunk L % 8. VARIANT
// makes the type unique to each kernel instantiation (see Bf16Dma for why).
template <class T, int VARIANT>
struct Int8Dma {
    rsrc_t ra, rw;
    uint32_t off[T::IPW];
    int wave, chunk_byte, K;
    uint8_t *smem;

    __device__ __forceinline__ Int8Dma(const Int8Args &g, const int8_t *w, int64_t m0, int64_t m1, int64_t n0,
                                       int wave_, int lane, uint8_t *smem_)
        : wave(wave_), K((int)g.K), smem(smem_) {
        const int sub = lane >> 3;
        const int64_t mrows = m1 - m0 < T::BM ? m1 - m0 : T::BM, nrows = g.N - n0 < T::BN ? g.N - n0 : T::BN;
        rw = make_rsrc(w + n0 * K, nrows * K);
        ra = g.rows ? make_rsrc(g.a, g.tokens * K) : make_rsrc(g.a + m0 * K, mrows * K);
        chunk_byte = swz_chunk(sub, lane & 7) << 4;   // (tile rows 8 i + sub: their swizzle is sub's)
#pragma unroll
        for (int t = 0; t < T::IPW; ++t) {
            const int tt = t < T::A_INSTR ? t : t - T::A_INSTR;
            const int row = 8 * (T::NW * tt + wave) + sub;
            if (t < T::A_INSTR && g.rows) {
                const int token = row < mrows ? g.rows[m0 + row] : -1;
                off[t] = token >= 0 && token < g.tokens ? (uint32_t)token * (uint32_t)K + chunk_byte : kNowhere;
            } else {
                off[t] = (uint32_t)(row * K) + chunk_byte;
            }
        }
    }

    // the copies of K step ks into its stage buffer. Bytes of W past K read as zero, which
    // makes what A holds there (the next row's bytes) count for nothing.
    __device__ __forceinline__ void issue(int ks) const {
        uint8_t *base = smem + (ks % T::NSTAGE) * T::STAGE;
        const int koff = __builtin_amdgcn_readfirstlane(ks * KB);
        const bool past = koff + chunk_byte >= K;
#pragma unroll
        for (int t = 0; t < T::IPW; ++t) {
            if (t < T::A_INSTR)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void *)(base + 8 * (T::NW * t + wave) * KB), 16,
                                                         past ? kNowhere : off[t], koff, 0, 0);
            else
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    rw, (lds_void *)(base + T::A_BYTES + 8 * (T::NW * (t - T::A_INSTR) + wave) * KB), 16,
                    past ? kNowhere : off[t], koff, 0, 0);
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

template <int BM_, int BN_, int NW_, int WAVES_M_, int OUT_BF16, int GROUPED>
__global__ __launch_bounds__(NW_ * 64) __attribute__((amdgpu_waves_per_eu(2, 2))) void int8_tile_kernel(Int8Args g) {
    using T = Int8Tile<BM_, BN_, NW_, WAVES_M_>;
    constexpr int SUB_M = T::SUB_M, SUB_N = T::SUB_N, WM = T::WM, WN = T::WN;
    __shared__ __attribute__((aligned(16))) uint8_t smem[T::STAGE * T::NSTAGE];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave % T::WAVES_M, wn = wave / T::WAVES_M;

    // XCD-contiguous tile index (workgroup b runs on XCD b % 8), then down `group` tile rows
    // per tile column
    const int tiles = g.tiles_m * g.tiles_n;
    const int xcd = blockIdx.x & 7, slot = blockIdx.x >> 3;
    const int q = tiles >> 3, rem = tiles & 7;
    const int tl = xcd * q + (xcd < rem ? xcd : rem) + slot;
    const int band = tl / (g.group * g.tiles_n);
    const int in_band = tl - band * g.group * g.tiles_n;
    const int band_rows = min(g.group, g.tiles_m - band * g.group);
    const int tile_m = band * g.group + in_band % band_rows;
    const int64_t n0 = (int64_t)(in_band / band_rows) * T::BN;
    int64_t m0, m1;
    const int8_t *w = g.w;
    const float *sw = g.sw;
    if constexpr (GROUPED) {
        int expert;
        if (!find_block(g, T::BM, tile_m, expert, m0, m1)) return;
        w += (int64_t)expert * g.N * g.K;
        sw += (int64_t)expert * g.N;
    } else {
        m0 = (int64_t)tile_m * T::BM;
        m1 = g.M;
    }
    const int nks = (int)((g.K + KB - 1) / KB);
    const Int8Dma<T, OUT_BF16 * 2 + GROUPED> dma(g, w, m0, m1, n0, wave, lane, smem);

    i32x4 acc[SUB_M][SUB_N];
#pragma unroll
    for (int i = 0; i < SUB_M; ++i)
#pragma unroll
        for (int j = 0; j < SUB_N; ++j) acc[i][j] = i32x4{0, 0, 0, 0};

    const int frow = lane & 15, kg = lane >> 4;
    const int lo = frow * KB + (swz_chunk(frow, kg) << 4);
    const int hi = frow * KB + (swz_chunk(frow, 4 + kg) << 4);
    const int a_base = wm * WM * KB, w_base = T::A_BYTES + wn * WN * KB;

    if (nks > 0) dma.issue(0);
    if (nks > 1) {
        dma.issue(1);
        wait_vmcnt<T::IPW>();
    } else {
        wait_vmcnt<0>();
    }
    lds_barrier();
    for (int ks = 0; ks < nks; ++ks) {
        const uint8_t *stage = smem + (ks & 1) * T::STAGE;
        u32x4 wf[SUB_N][2];
#pragma unroll
        for (int j = 0; j < SUB_N; ++j) {
            wf[j][0] = *reinterpret_cast<const u32x4 *>(stage + w_base + 16 * j * KB + lo);
            wf[j][1] = *reinterpret_cast<const u32x4 *>(stage + w_base + 16 * j * KB + hi);
        }
        u32x4 xa[2] = {*reinterpret_cast<const u32x4 *>(stage + a_base + lo),
                       *reinterpret_cast<const u32x4 *>(stage + a_base + hi)};
#pragma unroll
        for (int i = 0; i < SUB_M; ++i) {
            u32x4 xn[2] = {xa[0], xa[1]};
            if (i + 1 < SUB_M) {
                xn[0] = *reinterpret_cast<const u32x4 *>(stage + a_base + 16 * (i + 1) * KB + lo);
                xn[1] = *reinterpret_cast<const u32x4 *>(stage + a_base + 16 * (i + 1) * KB + hi);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < SUB_N; ++j) acc[i][j] = mfma_i8(wf[j][h], xa[h], acc[i][j]);
            xa[0] = xn[0];
            xa[1] = xn[1];
        }
        __builtin_amdgcn_sched_barrier(0);                                  // the waits stay behind this step's MFMAs
        __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (0 << 8) | (3 << 14));   // lgkmcnt(0)
        if (ks + 1 < nks) wait_vmcnt<0>();                                  // step ks + 1 has landed
        lds_barrier();
        if (ks + 2 < nks) dma.issue(ks + 2);
    }

    // Epilogue: scaled rows go through LDS and leave in whole 128-byte pieces (as in
    // bf16_gemm.hip), masked to the tile's rows and to N.
    using E = Int8Epilogue<T, OUT_BF16>;
    constexpr int OB = E::OB, EPC = E::EPC, LDS_ROW = E::LDS_ROW, RG = E::RG, IPR = E::IPR, CPR = E::CPR;
    const bool vec = ((g.N * OB) & 15) == 0 && (reinterpret_cast<uintptr_t>(g.y) & 15) == 0;
    f32x4 scale_n[SUB_N], bias[SUB_N];
#pragma unroll
    for (int j = 0; j < SUB_N; ++j) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int64_t n = n0 + wn * WN + 16 * j + 4 * kg + r;
            scale_n[j][r] = n < g.N ? sw[n] : 0.0f;
            bias[j][r] = g.bias && n < g.N ? g.bias[n] : 0.0f;
        }
    }
    float scale_m[SUB_M];
#pragma unroll
    for (int i = 0; i < SUB_M; ++i) {
        int64_t m = m0 + wm * WM + 16 * i + frow;
        scale_m[i] = 0.0f;
        if (m < m1) {
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
        for (int c = threadIdx.x; c < chunks; c += T::NW * 64) {
            const int r = c / CPR, cb = c - r * CPR;
            const int ii = r / RG, within = r - ii * RG;
            const int64_t m = m0 + (within >> 4) * WM + 16 * (i0 + ii) + (within & 15);
            const int64_t n = n0 + cb * EPC;
            if (m >= m1 || n >= g.N) continue;
            const uint8_t *src = smem + r * LDS_ROW + cb * 16;
            uint8_t *yp = reinterpret_cast<uint8_t *>(g.y) + (m * g.N + n) * OB;
            if (vec && n + EPC <= g.N) {
                *reinterpret_cast<u32x4 *>(yp) = *reinterpret_cast<const u32x4 *>(src);
            } else {
                for (int e = 0; e < EPC && n + e < g.N; ++e) {
                    if constexpr (OUT_BF16)
                        reinterpret_cast<uint16_t *>(yp)[e] = reinterpret_cast<const uint16_t *>(src)[e];
                    else
                        reinterpret_cast<float *>(yp)[e] = reinterpret_cast<const float *>(src)[e];
                }
            }
        }
    }
}

template <int MT, int U>
hipError_t launch_few(Int8Args a, bool out_bf16, hipStream_t stream) {
    a.tiles_n = (int)((a.N + 15) / 16);
    // grouped: an upper bound on the experts' row blocks (an expert without rows has none)
    int64_t blocks = (a.M + 16 * MT - 1) / (16 * MT);
    if (a.offsets) blocks += a.experts < a.M ? a.experts : a.M;
    const int64_t units = blocks * a.tiles_n;
    if (units * 256 > 0xFFFFFFFFll) return hipErrorInvalidValue;
    const dim3 grid((unsigned)units), block(256);
    if (a.offsets) {
        if (out_bf16) int8_few_kernel<MT, U, 1, 1><<<grid, block, 0, stream>>>(a);
        else int8_few_kernel<MT, U, 0, 1><<<grid, block, 0, stream>>>(a);
    } else {
        if (out_bf16) int8_few_kernel<MT, U, 1, 0><<<grid, block, 0, stream>>>(a);
        else int8_few_kernel<MT, U, 0, 0><<<grid, block, 0, stream>>>(a);
    }
    return hipGetLastError();
}

template <int BM, int BN, int NW, int WAVES_M>
hipError_t launch_tile(Int8Args a, bool out_bf16, hipStream_t stream) {
    a.tiles_m = (int)((a.M + BM - 1) / BM + (a.offsets ? (a.experts < a.M ? a.experts : a.M) : 0));
    a.tiles_n = (int)((a.N + BN - 1) / BN);
    // tile rows walked per tile column: an XCD's ~32 resident tiles form a compact block
    int64_t best = -1;
    for (int gsz = 1; gsz <= 32; gsz *= 2) {
        const int64_t gg = gsz < a.tiles_m ? gsz : a.tiles_m, cols = (32 + gg - 1) / gg;
        const int64_t rows = gg * BM + (cols < a.tiles_n ? cols : a.tiles_n) * BN;
        if (best < 0 || rows < best) {
            best = rows;
            a.group = gsz;
        }
    }
    const int64_t tiles = (int64_t)a.tiles_m * a.tiles_n;
    if (tiles * NW * 64 > 0xFFFFFFFFll) return hipErrorInvalidValue;
    const dim3 grid((unsigned)tiles), block(NW * 64);
    if (a.offsets) {
        if (out_bf16) int8_tile_kernel<BM, BN, NW, WAVES_M, 1, 1><<<grid, block, 0, stream>>>(a);
        else int8_tile_kernel<BM, BN, NW, WAVES_M, 0, 1><<<grid, block, 0, stream>>>(a);
    } else {
        if (out_bf16) int8_tile_kernel<BM, BN, NW, WAVES_M, 1, 0><<<grid, block, 0, stream>>>(a);
        else int8_tile_kernel<BM, BN, NW, WAVES_M, 0, 0><<<grid, block, 0, stream>>>(a);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_int8_quant(const uint16_t *x, int8_t *q, float *s, int64_t M, int64_t K, hipStream_t stream) {
    const dim3 block(256), four((unsigned)((M + 3) / 4)), one((unsigned)M);
    if (K <= 512) row_quant_kernel<1, 1><<<four, block, 0, stream>>>(x, q, s, M, K);
    else if (K <= 2048) row_quant_kernel<1, 4><<<four, block, 0, stream>>>(x, q, s, M, K);
    else if (K <= 8192) row_quant_kernel<4, 4><<<one, block, 0, stream>>>(x, q, s, M, K);
    else if (K <= 32768) row_quant_kernel<4, 16><<<one, block, 0, stream>>>(x, q, s, M, K);
    else row_quant_kernel<4, 0><<<one, block, 0, stream>>>(x, q, s, M, K);
    return hipGetLastError();
}

hipError_t launch_int8_gemm(const int8_t *a, const float *sa, const int8_t *w, const float *sw, const float *bias,
                            void *y, bool out_bf16, int64_t M, int64_t N, int64_t K, hipStream_t stream) {
    const Int8Args g{a, sa, w, sw, bias, y, nullptr, nullptr, M, N, K, M, 0, 0, 0, 1};
    if (M <= 16) return launch_few<1, 8>(g, out_bf16, stream);
    if (M <= 32) return launch_few<2, 4>(g, out_bf16, stream);
    if (M <= 64) return launch_few<4, 4>(g, out_bf16, stream);
    const int64_t large = ((M + 255) / 256) * ((N + 255) / 256);
    if (large >= 256) return launch_tile<256, 256, 8, 2>(g, out_bf16, stream);
    return launch_tile<128, 128, 4, 2>(g, out_bf16, stream);
}

hipError_t launch_int8_grouped_gemm(const int8_t *a, const float *sa, const int8_t *w, const float *sw,
                                    const int64_t *offsets, const int32_t *rows, void *y, bool out_bf16,
                                    int64_t experts, int64_t M, int64_t tokens, int64_t N, int64_t K,
                                    hipStream_t stream) {
    const Int8Args g{a, sa, w, sw, nullptr, y, offsets, rows, M, N, K, tokens, (int)experts, 0, 0, 1};
    if (M <= 16 * experts) return launch_few<1, 8>(g, out_bf16, stream);
    return launch_tile<128, 128, 4, 2>(g, out_bf16, stream);
}

}  // namespace fp8q
