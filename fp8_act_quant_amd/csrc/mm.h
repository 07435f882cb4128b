// mm.h -- tiles of bf16 products for gfx950, shared by the gated projections (gated.hip) and the
// adapters (adapter.hip): acc[m, n] = sum_k X(m, k) W(n, k), products exact in fp32, summed in fp32 by
// v_mfma_f32_16x16x32_bf16.
//
// Operands. Each of X and W is rows of K ("x[m, k]", K contiguous) or columns of it ("x[k, m]", K
// strided): y = x w^T reads both in the first way, the gradient of x reads W in the second, that of the
// weight both. A K-contiguous operand lies in LDS as rows of 64 k (128 bytes), 16-byte chunk c of row r
// at c ^ (r & 7); a K-strided one as panels of 64 k-rows x 128 columns (or 64), as it is in memory, and is
// transposed by its LDS reads (ds_read_b64_tr_b16: 16 lanes read 4 k-rows x 16 columns and each gets one
// column's 4), with the 32-byte pieces of a k-row exchanged by its number, so that neither kind of read
// meets a bank conflict. (Passes that transpose them first move 302 MB in a gradient of 4096 x 7168 -> 2048:
// 59 us at a copy's rate beside its 400.)
//
// Orientation. W is the MFMA's A operand and X its B operand: lane l of a 16 x 16 result holds
// n = 4 * (l / 16) + r (r = 0..3) for m = l % 16, four consecutive outputs of a row of Y. A lane's
// operands are 8 consecutive k at 32 h + 8 * (l / 16), h = 0, 1 within a step of 64.
//
// GATED: W is [2 F, K], and the columns of a wave are half of them gate columns and half the up
// columns of the same f, so that the product of the two halves needs no exchange.
//
// What lies past K, M or N is read as zeros (beyond the range of a buffer resource, or at an offset
// made so); both operands are zero past K, so that nothing there, not even NaN, reaches a sum.
#pragma once

#include "device_common.h"
#include "launch.h"

namespace fp8q {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __amdgpu_buffer_rsrc_t rsrc_t;
// memory at the alignment of an element
typedef u32x4 __attribute__((aligned(2))) u32x4_any;
typedef u32x2 __attribute__((aligned(2))) u32x2_any;

constexpr int KSTEP = 64, KB = 2 * KSTEP;   // elements and bytes of K in a step
constexpr uint32_t kNowhere = 0xFFFFFFF0u;  // an offset past every buffer's end: reads zeros

__device__ __forceinline__ rsrc_t make_rsrc(const void *p, int64_t bytes) {
    const uint32_t n = bytes > (int64_t)kNowhere ? kNowhere : bytes < 0 ? 0u : (uint32_t)bytes;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, (int)n, 0x00020000);
}

// The same resource as four words, and a copy of 16 bytes a lane from it to LDS (from `to` on, a wave's 1 KB) of which
// the compiler does not know: with one that it knows of, it waits for all copies under way before every transposing
// LDS read (4096 x 7168 x 4096 by 128 x 128 tiles 600 us instead of 240). The waits here are written out anyway, and
// those that the compiler adds for loads of its own only get longer.
__device__ __forceinline__ u32x4 rsrc_words(const void *p, int64_t bytes) {
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    return u32x4{(uint32_t)a, (uint32_t)(a >> 32) & 0xFFFFu, bytes > (int64_t)kNowhere ? kNowhere : bytes < 0 ? 0u : (uint32_t)bytes,
                 0x00020000u};
}
__device__ __forceinline__ void copy16(const u32x4 &rsrc, uint8_t *to, uint32_t off, uint32_t soff) {
    const uint32_t lds = (uint32_t)(uintptr_t)(lds_void *)to;
    uint32_t m0;   // (M0 is put back: the compiler, which takes no clobber of it, may hold a value of its own there)
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %3, %4 offen lds\n\ts_mov_b32 m0, %0"
                 : "=&s"(m0)
                 : "s"(lds), "v"(off), "s"(rsrc), "s"(soff)
                 : "memory");
}

__device__ __forceinline__ int swz_chunk(int row, int chunk) { return chunk ^ (row & 7); }

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}
__device__ __forceinline__ void wait_lgkm0() { __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (0 << 8) | (3 << 14)); }

__device__ __forceinline__ void lds_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

__device__ __forceinline__ f32x4 mfma_bf16(const u32x4 &w, const u32x4 &x, f32x4 acc) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, x), acc,
                                                   0, 0, 0);
}

// Tiles of BM x BN, NW waves in a WAVES_M x (NW / WAVES_M) grid. Tile rows go to the waves in groups of 16
// in turn: group i of the waves in row wm of the grid starts at tile row row(wm, i), so of 256 rows the
// first 128 are every wave's first half.
template <int BM_, int BN_, int NW_, int WAVES_M_, int NSTAGE_>
struct Tile {
    static constexpr int BM = BM_, BN = BN_, NW = NW_, WAVES_M = WAVES_M_, WAVES_N = NW_ / WAVES_M_;
    static constexpr int NSTAGE = NSTAGE_;
    static constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N;
    static constexpr int SUB_M = WM / 16, SUB_N = WN / 16;
    static constexpr int X_BYTES = BM * KB, W_BYTES = BN * KB, STAGE = X_BYTES + W_BYTES;
    static constexpr int X_INSTR = BM / (8 * NW), W_INSTR = BN / (8 * NW), IPW = X_INSTR + W_INSTR;
    static constexpr int PX = BM < 128 ? BM : 128, PW = BN < 128 ? BN : 128;   // columns of a panel
    static_assert(WAVES_M * WAVES_N == NW && BM % (8 * NW) == 0 && BN % (8 * NW) == 0, "tile shape");
    static_assert(STAGE * NSTAGE <= 160 * 1024 && IPW * (NSTAGE - 1) < 64, "LDS budget, vmcnt range");
    __device__ static __forceinline__ constexpr int group(int wm, int i) { return i * WAVES_M + wm; }
    __device__ static __forceinline__ constexpr int row(int wm, int i) { return 16 * group(wm, i); }
};

struct MmArgs {
    const uint16_t *x, *w;
    int64_t M, N, K;      // rows and columns of the output (GATED: N = F), depth
    int64_t ldx, ldw;     // elements from a row (K contiguous) or from a k (K strided) to the next
    int tiles_m, tiles_n, group;
};

// The m and n of tile number `tile`
__device__ __forceinline__ void place_tile(const MmArgs &g, int tile, int bm, int bn, int64_t &m0, int64_t &n0) {
    const int band = tile / (g.group * g.tiles_n);
    const int in_band = tile - band * g.group * g.tiles_n;
    const int band_rows = min(g.group, g.tiles_m - band * g.group);
    m0 = (int64_t)(band * g.group + in_band % band_rows) * bm;
    n0 = (int64_t)(in_band / band_rows) * bn;
}

// Workgroup b's tile. Workgroups are dealt round-robin to the 8 XCDs; each XCD takes a contiguous run of
// the tile numbers, which go down `group` tile rows per tile column, so that the tiles that an XCD holds
// at once share panels in its L2. NT: columns of Y in a tile.
template <class T, int NT>
__device__ __forceinline__ void find_tile(const MmArgs &g, int64_t &m0, int64_t &n0) {
    const int tiles = g.tiles_m * g.tiles_n;
    const int xcd = blockIdx.x & 7, slot = blockIdx.x >> 3;
    const int q = tiles >> 3, rem = tiles & 7;
    place_tile(g, xcd * q + (xcd < rem ? xcd : rem) + slot, T::BM, NT, m0, n0);
}

// The largest tiles, of one product or of two independent ones of n_a and n_b tiles, one a CU: each XCD takes a
// contiguous run of a's and one of b's. Where they are more than its 32 CUs take at once and the last round has
// at most 16, that round's tiles are cut into halves of 128 rows for twice the CUs (896 tiles of 256 x 256: 3.5 rounds
// instead of 4, a 12th of the time). Returns false where a workgroup has none; half: -1 (whole), 0 or 1.
__host__ __device__ __forceinline__ int run_of(int n, int xcd) { return (int)((int64_t)n * xcd / 8); }
__host__ __device__ __forceinline__ int whole_of(int total) {
    const int last = total & 31;
    return total > 32 && last <= 16 ? total - last : total;
}
__device__ __forceinline__ bool find_share(int n_a, int n_b, bool &second, int &tile, int &half) {
    const int xcd = blockIdx.x & 7, slot = blockIdx.x >> 3;
    const int a0 = run_of(n_a, xcd), b0 = run_of(n_b, xcd), a = run_of(n_a, xcd + 1) - a0, total = a + run_of(n_b, xcd + 1) - b0;
    const int whole = whole_of(total);
    int at = slot;
    half = -1;
    if (slot >= whole) at = whole + (slot - whole) / 2, half = (slot - whole) & 1;
    second = at >= a;
    tile = second ? b0 + at - a : a0 + at;
    return at < total;
}
inline unsigned share_grid(int n_a, int n_b) {
    int most = 0;
    for (int xcd = 0; xcd < 8; ++xcd) {
        const int total = run_of(n_a, xcd + 1) - run_of(n_a, xcd) + run_of(n_b, xcd + 1) - run_of(n_b, xcd);
        const int slots = 2 * total - whole_of(total);
        most = slots > most ? slots : most;
    }
    return 8 * (unsigned)most;
}
// A product's time (us) by its tiles: rounds of 256 of them (one a CU), each an epilogue and K's steps, of which a later
// round's may hide behind the round before. halves: the last round may be half a one. It ranks tiles. What is the same for
// all of them is not in it: the read of W from memory (48 x 7168 x 7168 comes out at 17 us and takes 30), adapters, the kind
// of epilogue (a gated projection's kept ones, fp32 outputs).
inline double tile_time(int64_t M, int64_t N, int64_t steps, int bm, int bn, double first, double more, double end, bool halves) {
    const double n = (double)((M + bm - 1) / bm) * (double)((N + bn - 1) / bn);
    if (n > 4e6) return halves ? 1e30 : 1e31;   // (a grid holds 2^32 threads; the largest tiles have the fewest)
    const int64_t whole = (int64_t)n / 256, last = (int64_t)n % 256;
    const double rounds = (double)whole + (last == 0 ? 0.0 : halves && whole > 0 && last <= 128 ? 0.6 : 1.0);
    return (double)steps * (first + more * (rounds - 1.0)) + end * rounds;
}
using WholeTile = Tile<256, 256, 8, 2, 2>;
using HalfTile = Tile<128, 256, 8, 2, 3>;

// The most workgroups of `threads` threads in a grid, which holds 2^32 - 1 threads
constexpr int64_t grid_limit(int threads) { return 0xFFFFFFFFll / threads; }
// Workgroups of share_grid beyond the tiles: 16 halves an XCD, and XCDs of one or two tiles fewer than another
constexpr int64_t kShareMore = 8 * 18;

// The tiles of a launch, and down how many tile rows to walk (so that the some 32 tiles of an XCD read the
// fewest rows of both operands). False: more than a grid holds, `more` workgroups beside the tiles.
inline bool lay_out(MmArgs &a, int bm, int bn, int threads, int64_t more = 0) {
    const int64_t tm = (a.M + bm - 1) / bm, tn = (a.N + bn - 1) / bn;
    a.tiles_m = a.tiles_n = 0;
    if (tm == 0 || tn == 0) return true;
    const int64_t most = grid_limit(threads) - more;
    if (tm > most || tn > most || tm > most / tn) return false;
    a.tiles_m = (int)tm;
    a.tiles_n = (int)tn;
    int64_t best = -1;
    for (int g = 1; g <= 32; g *= 2) {
        const int64_t gg = g < tm ? g : tm, cols = (32 + gg - 1) / gg, rows = gg * bm + (cols < tn ? cols : tn) * bn;
        if (best < 0 || rows < best) best = rows, a.group = g;
    }
    return true;
}

// The exchange of 32-byte pieces in k-row `row` of a panel of P columns: with rows of 256 bytes (8 pieces)
// by the bits that tell apart the 8 rows that 32 lanes read, with rows of 128 bytes (4 pieces), two of
// which lie side by side in the banks, by two of them
template <int P>
__device__ __forceinline__ int exchange(int row) {
    return P == 128 ? (row & 3) | (row >> 1 & 4) : (row >> 1 & 1) | (row >> 2 & 2);
}

// This wave's copies global -> LDS (LDS-DMA, 1 KB each): instruction q = NW t + wave of an operand fills
// the q-th KB of its part of a stage, with 8 rows of a K-contiguous operand or 1024 / (2 P) k-rows of a
// panel of a K-strided one. XT, WT: the operand is K-strided. TAG makes the type unique to each kernel
// instantiation: the host pass emits a launch stub for only one kernel among those that share such a type.
template <class T, int XT, int WT, int GATED, int TAG>
struct Copies {
    rsrc_t rx, rw, rw1;               // K-contiguous (GATED: rw1 the up rows)
    u32x4 rxw;                        // rx where an operand is K-strided
    const uint16_t *px, *pw;          // K-strided: column m0, n0 of k-row 0
    int64_t left_x, left_w;           // their bytes from there to the operand's end
    uint32_t off[T::IPW];
    int64_t ldx, ldw;
    int wave, chunk_byte, Kb;

    __device__ __forceinline__ int instr(int t) const { return T::NW * (t < T::X_INSTR ? t : t - T::X_INSTR) + wave; }
    // GATED: whether W's instruction t copies up rows (the same for all lanes: a wave's columns are 16 or
    // more of each kind in a row, an instruction 8)
    __device__ __forceinline__ bool up(int t) const { return 8 * instr(t) % T::WN >= T::WN / 2; }

    template <int P>
    __device__ static __forceinline__ uint32_t strided(int q, int lane, int64_t ld) {
        constexpr int PER = P / 8;    // copies of a panel, chunks of a k-row
        const int panel = q / PER, row = (q % PER) * (512 / P) + lane / PER, chunk = lane % PER;
        const int piece = (chunk >> 1) ^ exchange<P>(row);
        return (uint32_t)(row * ld * 2) + 2 * (panel * P + 16 * piece + 8 * (chunk & 1));
    }

    __device__ __forceinline__ Copies(const MmArgs &g, int64_t m0, int64_t n0, int wave_, int lane)
        : ldx(g.ldx), ldw(g.ldw), wave(wave_), Kb((int)(2 * g.K)) {
        const int sub = lane >> 3;
        chunk_byte = swz_chunk(sub, lane & 7) << 4;   // (rows 8 i + sub: their swizzle is sub's)
        if constexpr (XT) {
            px = g.x + m0;
            left_x = 2 * (g.K * ldx - m0);
        } else {
            const int64_t rows = g.M - m0 < T::BM ? g.M - m0 : T::BM;
            rx = make_rsrc(g.x + m0 * ldx, 2 * ((rows - 1) * ldx + g.K));
            rxw = rsrc_words(g.x + m0 * ldx, 2 * ((rows - 1) * ldx + g.K));
        }
        if constexpr (WT) {
            pw = g.w + n0;
            left_w = 2 * (g.K * ldw - n0);
        } else {
            const int64_t most = GATED ? T::BN / 2 : T::BN, rows = g.N - n0 < most ? g.N - n0 : most;
            rw = make_rsrc(g.w + n0 * ldw, 2 * ((rows - 1) * ldw + g.K));
            if constexpr (GATED) rw1 = make_rsrc(g.w + (g.N + n0) * ldw, 2 * ((rows - 1) * ldw + g.K));
        }
#pragma unroll
        for (int t = 0; t < T::IPW; ++t) {
            const int q = instr(t);
            if (t < T::X_INSTR) {
                off[t] = XT ? strided<T::PX>(q, lane, ldx) : (uint32_t)((8 * q + sub) * ldx * 2) + chunk_byte;
            } else if (WT) {
                off[t] = strided<T::PW>(q, lane, ldw);
            } else {
                int row = 8 * q + sub;
                if (GATED) row = row / T::WN * (T::WN / 2) + row % (T::WN / 2);
                off[t] = (uint32_t)(row * ldw * 2) + chunk_byte;
            }
        }
    }

    // copies first .. first + count - 1 (X's, then W's; constants where this is inlined) of K step ks into
    // the stage at `base`; steps past the last copy zeros
    __device__ __forceinline__ void issue(uint8_t *base, int ks, int first = 0, int count = T::IPW) const {
        const int koff = __builtin_amdgcn_readfirstlane(ks * KB);
        const bool past = koff + chunk_byte >= Kb;
        u32x4 sx, sw;
        if constexpr (XT) sx = rsrc_words(px + ks * (KSTEP * ldx), left_x - ks * (KSTEP * 2 * ldx));
        if constexpr (WT) sw = rsrc_words(pw + ks * (KSTEP * ldw), left_w - ks * (KSTEP * 2 * ldw));
#pragma unroll
        for (int t = 0; t < T::IPW; ++t) {
            if (t < first || t >= first + count) continue;
            uint8_t *to = base + (t < T::X_INSTR ? 0 : T::X_BYTES) + 1024 * instr(t);
            if (t < T::X_INSTR) {
                if constexpr (XT) copy16(sx, to, off[t], 0);
                else if constexpr (WT) copy16(rxw, to, past ? kNowhere : off[t], koff);
                else __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_void *)to, 16, past ? kNowhere : off[t], koff, 0, 0);
            } else {
                if constexpr (WT) copy16(sw, to, off[t], 0);
                else if (GATED && up(t))
                    __builtin_amdgcn_raw_ptr_buffer_load_lds(rw1, (lds_void *)to, 16, past ? kNowhere : off[t], koff, 0, 0);
                else __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void *)to, 16, past ? kNowhere : off[t], koff, 0, 0);
            }
        }
    }
    static_assert(WT || !XT, "X alone is never K-strided");
};

// This wave's operands from a stage: half h (32 k) of its 16-row group i of X, or 16-column block j of W
template <class T, int XT, int WT>
struct Operands {
    static constexpr int BX = T::PX / 16, BW = T::PW / 16;   // blocks of a panel
    static constexpr int XV = XT ? (T::SUB_M < BX / T::WAVES_M ? T::SUB_M : BX / T::WAVES_M) : 2;
    int x_at[XV], w_at[WT ? T::SUB_N : 2];

    template <int P>
    __device__ static __forceinline__ int strided(int block, int lane) {
        const int g = lane >> 4, q = (lane & 15) >> 2, row = 8 * g + q;   // (4 t and 32 h change no exchange)
        return row * (2 * P) + ((block ^ exchange<P>(row)) << 5) + (lane & 3) * 8;
    }
    __device__ __forceinline__ Operands(int lane, int wm, int wn) {
        const int row = lane & 15, kg = lane >> 4;
        const int lo = row * KB + (swz_chunk(row, kg) << 4), hi = row * KB + (swz_chunk(row, 4 + kg) << 4);
        if constexpr (XT) {
#pragma unroll
            for (int i = 0; i < XV; ++i) x_at[i] = strided<T::PX>(T::group(wm, i) % BX, lane);
        } else {
            x_at[0] = 16 * wm * KB + lo, x_at[1] = 16 * wm * KB + hi;
        }
        if constexpr (WT) {
            const int block = wn * T::SUB_N;
#pragma unroll
            for (int j = 0; j < T::SUB_N; ++j)
                w_at[j] = T::X_BYTES + (block / BW) * (KSTEP * 2 * T::PW) + strided<T::PW>(block % BW + j, lane);
        } else {
            w_at[0] = T::X_BYTES + wn * T::WN * KB + lo, w_at[1] = T::X_BYTES + wn * T::WN * KB + hi;
        }
    }
    template <int P>
    __device__ static __forceinline__ u32x4 transposed(const uint8_t *p, int h) {
        u32x4 v;
        const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + h * 32 * 2 * P));
        const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + (h * 32 + 4) * 2 * P));
        const u32x2 ua = __builtin_bit_cast(u32x2, a), ub = __builtin_bit_cast(u32x2, b);
        v[0] = ua[0], v[1] = ua[1], v[2] = ub[0], v[3] = ub[1];
        return v;
    }
    __device__ __forceinline__ u32x4 x(const uint8_t *stage, int i, int h) const {
        if constexpr (XT)   // (a panel's groups are the waves' in turn)
            return transposed<T::PX>(stage + i / XV * (KSTEP * 2 * T::PX) + x_at[i % XV], h);
        else return *reinterpret_cast<const u32x4 *>(stage + x_at[h] + i * (16 * T::WAVES_M * KB));
    }
    __device__ __forceinline__ u32x4 w(const uint8_t *stage, int j, int h) const {
        if constexpr (WT) return transposed<T::PW>(stage + w_at[j], h);
        else return *reinterpret_cast<const u32x4 *>(stage + w_at[h] + 16 * j * KB);
    }
};

// Tiles of 8 waves, two to a SIMD, that take turns: waves 0-3 and 4-7 are one barrier apart, so that in
// each interval between two barriers ("slot") one wave of a SIMD multiplies from registers while the
// other fills its own from LDS and queues copies. A wave's K step is PH phases (2 for BM = 256, 1 for
// 128), each a load slot and a multiply slot of 32 MFMAs: phase 0 loads the step's W operands and the
// wave's first 64 rows of X, phase 1 the other 64 rows, over the same registers.
//
// Copies. A region of a stage is free once both groups have loaded it, which each load slot ends by
// waiting for (lgkmcnt). With two phases and two stages, the copies of step ks + 2 for W and the tile's
// first 128 rows are queued in load slot 1 of step ks, those of its other rows in load slot 0 of step
// ks + 1; with one phase and three stages, those of step ks + 2 in the load slot of step ks. Copies
// retire in order, and the count left open at the end of each load slot (IPW) covers exactly what the
// load slots before the data's use have queued since; the barrier then makes it visible. Steps past the
// last copy zeros, which keeps the counts the same.
template <class T, int XT, int WT, int GATED, int TAG, class F>
__device__ __forceinline__ void turns(const MmArgs &g, int64_t m0, int64_t n0, uint8_t *smem,
                                      f32x4 (&acc)[T::SUB_M][T::SUB_N], const F &begin) {
    constexpr int SUB_M = T::SUB_M, SUB_N = T::SUB_N, PH = SUB_M / 4;
    static_assert(T::NW == 8 && T::WAVES_M == 2 && (PH == 1 || PH == 2) && T::NSTAGE == 4 - PH, "schedule");
    constexpr int X0 = T::X_INSTR / 2;   // two phases: copies of the first 128 rows
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nks = (int)((g.K + KSTEP - 1) / KSTEP);
    const Copies<T, XT, WT, GATED, TAG> copies(g, m0, n0, wave, lane);
    const Operands<T, XT, WT> from(lane, wave >> 2, wave & 3);

#pragma unroll
    for (int i = 0; i < SUB_M; ++i)
#pragma unroll
        for (int j = 0; j < SUB_N; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    if constexpr (PH == 2) {
        copies.issue(smem, 0, T::X_INSTR, T::W_INSTR);
        copies.issue(smem, 0, 0, X0);
        copies.issue(smem, 0, X0, X0);
        copies.issue(smem + T::STAGE, 1, T::X_INSTR, T::W_INSTR);
        copies.issue(smem + T::STAGE, 1, 0, X0);
    } else {
        copies.issue(smem, 0);
        copies.issue(smem + T::STAGE, 1);
    }
    begin();
    __builtin_amdgcn_sched_barrier(0);
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
                for (int j = 0; j < SUB_N; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h) wf[j][h] = from.w(stage, j, h);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) xf[i][h] = from.x(stage, 4 * ph + i, h);
            if constexpr (PH == 1) {
                copies.issue(stage2, ks + 2);
            } else if (ph == 0) {
                copies.issue(stage1, ks + 1, X0, X0);
            } else {
                copies.issue(stage2, ks + 2, T::X_INSTR, T::W_INSTR);
                copies.issue(stage2, ks + 2, 0, X0);
            }
            __builtin_amdgcn_sched_barrier(0);   // the waits stay behind the loads and copies
            wait_lgkm0();
            wait_vmcnt<T::IPW>();
            lds_barrier();
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < SUB_N; ++j)
                        acc[4 * ph + i][j] = mfma_bf16(wf[j][h], xf[i][h], acc[4 * ph + i][j]);
            __builtin_amdgcn_s_setprio(0);
            __builtin_amdgcn_sched_barrier(0);
            lds_barrier();
        }
        stage = stage1;
        stage1 = stage2;
    }
    if (wave < 4) lds_barrier();
    wait_vmcnt<0>();   // the copies past the last step, before LDS takes something else
    __syncthreads();
}

// Smaller tiles of 4 waves, for shapes with too few of the large ones: their time is K's steps one after
// another, each waiting for memory, so as many stages as fit are in flight. Two register sets hold the
// operands of two steps: the MFMAs of step ks take one while the other is filled with step ks + 1, each
// row group's preceded by its share of the LDS reads and copies. A stage is free once its step is in
// registers everywhere (lgkmcnt, then the barrier), and takes the copies of step ks + NSTAGE; steps past the
// last copy zeros, so that the count left open always covers NSTAGE - 2 steps.
template <class T, int XT, int WT, int GATED, int TAG, class F>
__device__ __forceinline__ void deep(const MmArgs &g, int64_t m0, int64_t n0, uint8_t *smem,
                                     f32x4 (&acc)[T::SUB_M][T::SUB_N], const F &begin) {
    constexpr int SUB_M = T::SUB_M, SUB_N = T::SUB_N, READS = 2 * (SUB_M + SUB_N), GROUPS = 2 * SUB_M;
    static_assert(T::NW == 4 && T::WAVES_M == 2 && T::NSTAGE >= 3, "schedule");
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nks = (int)((g.K + KSTEP - 1) / KSTEP);
    const Copies<T, XT, WT, GATED, TAG> copies(g, m0, n0, wave, lane);
    const Operands<T, XT, WT> from(lane, wave & 1, wave >> 1);

#pragma unroll
    for (int i = 0; i < SUB_M; ++i)
#pragma unroll
        for (int j = 0; j < SUB_N; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < T::NSTAGE; ++s) copies.issue(smem + s * T::STAGE, s);
    begin();
    __builtin_amdgcn_sched_barrier(0);
    wait_vmcnt<T::IPW *(T::NSTAGE - 1)>();
    lds_barrier();
    u32x4 wf0[SUB_N][2], xf0[SUB_M][2], wf1[SUB_N][2], xf1[SUB_M][2];
    auto read = [&](const uint8_t *stage, int r, u32x4(&wf)[SUB_N][2], u32x4(&xf)[SUB_M][2]) {
        if (r / 2 < SUB_N) wf[r / 2][r & 1] = from.w(stage, r / 2, r & 1);
        else xf[r / 2 - SUB_N][r & 1] = from.x(stage, r / 2 - SUB_N, r & 1);
    };
#pragma unroll
    for (int r = 0; r < READS; ++r) read(smem, r, wf0, xf0);
    auto step = [&](int ks, uint8_t *stage, const uint8_t *stage1, const u32x4(&wf)[SUB_N][2],
                    const u32x4(&xf)[SUB_M][2], u32x4(&wn)[SUB_N][2], u32x4(&xn)[SUB_M][2]) {
        __builtin_amdgcn_sched_barrier(0);            // the waits stay behind the previous step's MFMAs
        wait_lgkm0();                                 // step ks is in registers
        wait_vmcnt<T::IPW *(T::NSTAGE - 2)>();        // step ks + 1 has landed
        lds_barrier();
#pragma unroll
        for (int q = 0; q < GROUPS; ++q) {
#pragma unroll
            for (int r = q * READS / GROUPS; r < (q + 1) * READS / GROUPS; ++r) read(stage1, r, wn, xn);
#pragma unroll
            for (int c = q * T::IPW / GROUPS; c < (q + 1) * T::IPW / GROUPS; ++c)
                copies.issue(stage, ks + T::NSTAGE, c, 1);
            const int h = q / SUB_M, i = q % SUB_M;
#pragma unroll
            for (int j = 0; j < SUB_N; ++j) acc[i][j] = mfma_bf16(wf[j][h], xf[i][h], acc[i][j]);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    uint8_t *const end = smem + T::NSTAGE * T::STAGE;
    uint8_t *stage = smem;
    for (int ks = 0; ks < nks; ks += 2) {
        // (with an odd number of steps the last one here multiplies zeros)
        uint8_t *stage1 = stage + T::STAGE == end ? smem : stage + T::STAGE;
        uint8_t *stage2 = stage1 + T::STAGE == end ? smem : stage1 + T::STAGE;
        step(ks, stage, stage1, wf0, xf0, wf1, xf1);
        step(ks + 1, stage1, stage2, wf1, xf1, wf0, xf0);
        stage = stage2;
    }
    wait_lgkm0();
    wait_vmcnt<0>();   // the copies past the last step, before LDS takes something else
    __syncthreads();
}

// `begin` is called once the first copies are on their way; it may put something into acc, or load
template <class T, int XT, int WT, int GATED, int TAG, class F>
__device__ __forceinline__ void multiply(const MmArgs &g, int64_t m0, int64_t n0, uint8_t *smem,
                                         f32x4 (&acc)[T::SUB_M][T::SUB_N], const F &begin) {
    if constexpr (T::NW == 8) turns<T, XT, WT, GATED, TAG>(g, m0, n0, smem, acc, begin);
    else deep<T, XT, WT, GATED, TAG>(g, m0, n0, smem, acc, begin);
}
template <class T>
__device__ __forceinline__ int wave_m() {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    return T::NW == 8 ? wave >> 2 : wave & 1;
}
template <class T>
__device__ __forceinline__ int wave_n() {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    return T::NW == 8 ? wave & 3 : wave >> 1;
}

// At most 16 RX rows (a decode step): every byte of W meets all of them once, so the read of W is what counts. A
// workgroup of 4 waves takes NB = 32 or 16 rows of W (GATED: half of them gate rows and half their up rows), which
// come through LDS with the rows of X, four steps of 64 k to a stage (a stage of one step costs a barrier and a wait for
// LDS as long as its copies). NB = 32: waves 0 and 1 take 16 rows of W each and the first half of every step, waves 2
// and 3 the other half. NB = 16, which gives the GPU twice the workgroups where W is small: each wave a step. The
// waves' sums are added in LDS: returns [row * NB + n] for row < 16 RX, the sums of X row `row` and the workgroup's row
// n of W (GATED: the gate rows first), for all to read. us with 32 / 16 rows: 1 x 7168 x 4096 11.0 / 10.5,
// 1 x 7168 x 1536 10.0 / 7.4.
template <int RX, int NB>
struct Few {
    static constexpr int ROWS = 16 * RX, SUBS = 4, STAGES = NB == 32 ? 3 : 5;
    static constexpr int W_SUB = NB * KB, X_SUB = ROWS * KB, STAGE = SUBS * (W_SUB + X_SUB), BYTES = STAGE * STAGES;
    static_assert(NB == 32 || NB == 16, "rows of W");
};
template <int RX, int NB, int GATED, int TAG, class F>
__device__ __forceinline__ const float *few(const MmArgs &g, int64_t n0, uint8_t *smem, const F &begin) {
    using P = Few<RX, NB>;
    constexpr int SUBS = P::SUBS, W_SUB = P::W_SUB, X_SUB = P::X_SUB, STAGE = P::STAGE, STAGES = P::STAGES;
    constexpr int W_EACH = NB / 8, IPW = W_EACH + 2 * RX;   // copies of a stage a wave: of W's 8-row pieces, of X's
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row = lane & 15, kg = lane >> 4, sub = lane >> 3;
    const int64_t most = GATED ? NB / 2 : NB, rows = g.N - n0 < most ? g.N - n0 : most;
    // W: a wave copies one 8-row piece of every step (NB = 32), or both of one (NB = 16)
    auto resource = [&](bool up) { return make_rsrc(g.w + (n0 + (up ? g.N : 0)) * g.ldw, 2 * ((rows - 1) * g.ldw + g.K)); };
    const rsrc_t rw = resource(GATED && NB == 32 && wave >= 2), rw1 = resource(GATED && NB == 16);
    const rsrc_t rx = make_rsrc(g.x, 2 * ((g.M - 1) * g.ldx + g.K));
    const int chunk_byte = swz_chunk(sub, lane & 7) << 4, Kb = (int)(2 * g.K);
    const int piece = NB == 32 ? (GATED ? wave & 1 : wave) : 0;
    const uint32_t w_off = (uint32_t)((8 * piece + sub) * g.ldw * 2) + chunk_byte;
    const uint32_t x_off = (uint32_t)(sub * g.ldx * 2) + chunk_byte, w_step = (uint32_t)(16 * g.ldw), x_step = (uint32_t)(16 * g.ldx);
    auto copy = [&](uint8_t *stage, int ks) {
        const int mine = __builtin_amdgcn_readfirstlane((ks * SUBS + wave) * KB);   // this wave's step
        const bool past = mine + chunk_byte >= Kb;
        if constexpr (NB == 32) {
#pragma unroll
            for (int s = 0; s < SUBS; ++s) {
                const int koff = __builtin_amdgcn_readfirstlane((ks * SUBS + s) * KB);
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void *)(stage + s * W_SUB + 1024 * wave), 16,
                                                         koff + chunk_byte >= Kb ? kNowhere : w_off, koff, 0, 0);
            }
        } else {
            lds_void *to = (lds_void *)(stage + wave * W_SUB), *to1 = (lds_void *)(stage + wave * W_SUB + 1024);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, to, 16, past ? kNowhere : w_off, mine, 0, 0);
            if constexpr (GATED) __builtin_amdgcn_raw_ptr_buffer_load_lds(rw1, to1, 16, past ? kNowhere : w_off, mine, 0, 0);
            else __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, to1, 16, past ? kNowhere : w_off + w_step, mine, 0, 0);
        }
#pragma unroll
        for (int t = 0; t < 2 * RX; ++t)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_void *)(stage + SUBS * W_SUB + wave * X_SUB + 1024 * t), 16,
                                                     past ? kNowhere : x_off + t * x_step, mine, 0, 0);
    };
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) copy(smem + s * STAGE, s);
    begin();
    __builtin_amdgcn_sched_barrier(0);
    const int cg = wave & 1, half = wave >> 1;
    const int lo = row * KB + (swz_chunk(row, kg) << 4), hi = row * KB + (swz_chunk(row, 4 + kg) << 4);
    const int nks = (int)((g.K + SUBS * KSTEP - 1) / (SUBS * KSTEP));
    f32x4 acc[RX];
#pragma unroll
    for (int i = 0; i < RX; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    uint8_t *stage = smem, *last = smem + (STAGES - 1) * STAGE;   // `last`: of the step before
    for (int ks = 0; ks < nks; ++ks) {
        __builtin_amdgcn_sched_barrier(0);
        wait_lgkm0();                         // the step before's reads
        wait_vmcnt<IPW *(STAGES - 2)>();      // this step has landed
        lds_barrier();
        copy(last, ks + STAGES - 1);
        auto multiply = [&](int s, int at, int w_base) {
            const u32x4 w = *reinterpret_cast<const u32x4 *>(stage + s * W_SUB + w_base + at);
#pragma unroll
            for (int i = 0; i < RX; ++i) {
                const u32x4 x = *reinterpret_cast<const u32x4 *>(stage + SUBS * W_SUB + s * X_SUB + 16 * i * KB + at);
                acc[i] = mfma_bf16(w, x, acc[i]);
            }
        };
        if constexpr (NB == 32) {
#pragma unroll
            for (int s = 0; s < SUBS; ++s) multiply(s, half ? hi : lo, 16 * cg * KB);
        } else {
            multiply(wave, lo, 0);
            multiply(wave, hi, 0);
        }
        last = stage;
        stage = stage + STAGE == smem + STAGES * STAGE ? smem : stage + STAGE;
    }
    wait_vmcnt<0>();
    __syncthreads();
    // Each wave's sums, as rows of X; then all of a sum's added
    constexpr int PARTS = NB == 32 ? 2 : 4, SIZE = P::ROWS * NB;
    static_assert(PARTS * SIZE * 4 <= P::BYTES, "LDS of the sums");
    float *const sums = reinterpret_cast<float *>(smem);
    float *const part = sums + (NB == 32 ? half : wave) * SIZE + (NB == 32 ? 16 * cg : 0) + 4 * kg;
#pragma unroll
    for (int i = 0; i < RX; ++i) *reinterpret_cast<f32x4 *>(part + (16 * i + row) * NB) = acc[i];
    __syncthreads();
    for (int p = threadIdx.x; p < SIZE / 4; p += 256) {
        f32x4 v = reinterpret_cast<const f32x4 *>(sums)[p];
#pragma unroll
        for (int q = 1; q < PARTS; ++q) v += reinterpret_cast<const f32x4 *>(sums + q * SIZE)[p];
        reinterpret_cast<f32x4 *>(sums)[p] = v;
    }
    __syncthreads();
    return sums;
}

// Four consecutive elements of a row with `left` of them from here on, as they are in memory
template <int BF16>
__device__ __forceinline__ f32x4 load4(const void *base, int64_t at, int64_t left) {
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    if constexpr (BF16) {
        const uint16_t *p = static_cast<const uint16_t *>(base) + at;
        if (left >= 4) {
            const u32x2 u = *reinterpret_cast<const u32x2_any *>(p);
            v = f32x4{bf16lo_to_f32(u[0]), bf16hi_to_f32(u[0]), bf16lo_to_f32(u[1]), bf16hi_to_f32(u[1])};
        } else {
#pragma unroll
            for (int r = 0; r < 3; ++r)
                if (r < left) v[r] = bf16lo_to_f32(p[r]);
        }
    } else {
        const float *p = static_cast<const float *>(base) + at;
        if (left >= 4) {
            v = __builtin_bit_cast(f32x4, *reinterpret_cast<const u32x4_any *>(p));
        } else {
#pragma unroll
            for (int r = 0; r < 3; ++r)
                if (r < left) v[r] = p[r];
        }
    }
    return v;
}
template <int BF16>
__device__ __forceinline__ void store4(void *base, int64_t at, const f32x4 &v, int64_t left) {
    if constexpr (BF16) {
        uint16_t *p = static_cast<uint16_t *>(base) + at;
        const u32x2 u = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        if (left >= 4) {
            *reinterpret_cast<u32x2_any *>(p) = u;
        } else {
#pragma unroll
            for (int r = 0; r < 3; ++r)
                if (r < left) p[r] = (uint16_t)(u[r / 2] >> (16 * (r & 1)));
        }
    } else {
        float *p = static_cast<float *>(base) + at;
        if (left >= 4) {
            *reinterpret_cast<u32x4_any *>(p) = __builtin_bit_cast(u32x4, v);
        } else {
#pragma unroll
            for (int r = 0; r < 3; ++r)
                if (r < left) p[r] = v[r];
        }
    }
}

// A tile's outputs, value(i, j) for its blocks, SUBS blocks of 16 columns a wave: they go through LDS and
// leave in whole 16-byte pieces, masked to M and N. (Stored straight from the registers each line would be
// written in 8-byte pieces by several instructions.) Begins and ends with a workgroup barrier.
template <class T, int BF16, int SUBS, class F>
__device__ __forceinline__ void store_tile(void *y, int64_t ldy, int64_t m0, int64_t M, int64_t n0, int64_t N,
                                           uint8_t *smem, const F &value) {
    constexpr int OB = BF16 ? 2 : 4, EPC = 16 / OB, COLS = T::WAVES_N * SUBS * 16;
    constexpr int ROW_WORDS = COLS * OB / 4, TARGET = BF16 ? 8 : 16;   // rows some banks apart
    constexpr int LDS_ROW = 4 * (ROW_WORDS + ((TARGET - ROW_WORDS) % 64 + 64) % 64);
    constexpr int RG = T::WAVES_M * 16, CPR = COLS * OB / 16;
    constexpr int IPR0 = T::STAGE * T::NSTAGE / (RG * LDS_ROW), IPR = IPR0 < T::SUB_M ? IPR0 : T::SUB_M;
    static_assert(IPR >= 1, "epilogue staging does not fit");
    const int lane = threadIdx.x & 63, wm = wave_m<T>(), wn = wave_n<T>();
    const int frow = lane & 15, kg = lane >> 4;
#pragma unroll
    for (int i0 = 0; i0 < T::SUB_M; i0 += IPR) {
        __syncthreads();
#pragma unroll
        for (int ii = 0; ii < IPR; ++ii) {
            if (i0 + ii < T::SUB_M) {
                uint8_t *rowp = smem + (ii * RG + wm * 16 + frow) * LDS_ROW;
#pragma unroll
                for (int j = 0; j < SUBS; ++j) {
                    const int col = 16 * (wn * SUBS + j) + 4 * kg;
                    const f32x4 v = value(i0 + ii, j);
                    if constexpr (BF16)
                        *reinterpret_cast<u32x2 *>(rowp + col * 2) =
                            u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
                    else
                        *reinterpret_cast<f32x4 *>(rowp + col * 4) = v;
                }
            }
        }
        __syncthreads();
        const int groups = (T::SUB_M - i0) < IPR ? (T::SUB_M - i0) : IPR;
        const int chunks = groups * RG * CPR;
        for (int c = threadIdx.x; c < chunks; c += T::NW * 64) {
            const int r = c / CPR, cb = c - r * CPR;
            const int ii = r / RG, within = r - ii * RG;
            const int64_t m = m0 + T::row(within >> 4, i0 + ii) + (within & 15);
            const int64_t n = n0 + cb * EPC;
            if (m >= M || n >= N) continue;
            const uint8_t *src = smem + r * LDS_ROW + cb * 16;
            uint8_t *yp = static_cast<uint8_t *>(y) + (m * ldy + n) * OB;
            if (n + EPC <= N) {
                *reinterpret_cast<u32x4_any *>(yp) = *reinterpret_cast<const u32x4 *>(src);
            } else {
                for (int e = 0; e < EPC && n + e < N; ++e) {
                    if constexpr (BF16)
                        reinterpret_cast<uint16_t *>(yp)[e] = reinterpret_cast<const uint16_t *>(src)[e];
                    else
                        reinterpret_cast<float *>(yp)[e] = reinterpret_cast<const float *>(src)[e];
                }
            }
        }
    }
    __syncthreads();
}

}  // namespace
}  // namespace fp8q
