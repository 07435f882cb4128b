// place.hip -- rows of a routed-expert layer into expert order, and back, for gfx950.
//
// moe_place: the T * k (token, choice) pairs, stably sorted by expert: offsets[e] .. offsets[e
// + 1] are expert e's rows, rows[r] the token of row r, slots[t, j] the row of token t's j-th
// choice. A counting sort: every workgroup owns a contiguous chunk of the pairs and each of
// its waves a contiguous segment of the chunk; counts per (wave, expert) are turned into first
// rows, and each wave then walks its segment 64 pairs at a time, a pair's row being its
// expert's next row plus the number of earlier lanes with the same expert. Nothing depends on
// the order in which waves or workgroups run. Integer work on a few hundred KB: what bounds it
// is the latency of its dependent steps, not bandwidth.
//
// moe_combine: y[t] = sum_j w[t, j] h[slots[t, j]], and its gradient. One pass over h, 16 bytes
// a lane; memory bound.
#include <cmath>

#include <fp8q.h>

#include "device_common.h"
#include "launch.h"

namespace fp8q {
namespace {

constexpr int kMaxExperts = (int)kMaxGroupedExperts;
constexpr int PW = 16;               // waves of a placement workgroup
constexpr int PT = 64 * PW;
// Pairs that one workgroup places by itself, in one launch (4096 pairs of 256 experts 5.5 us, 8192 9.3;
// two launches 7.3 and 7.5)
constexpr int64_t kOneChunk = 6144;
constexpr int64_t kChunk = 1024;    // pairs of a chunk where there are several
constexpr int64_t kMaxChunks = 256;

struct PlaceArgs {
    const int32_t *experts;
    int64_t *offsets;
    int32_t *rows;
    int32_t *slots;
    uint32_t *counts;   // [chunks][E]: each chunk's pairs of each expert
    int64_t pairs;
    int64_t seg;        // pairs of a wave, a multiple of 64
    int E, first, k, chunks;
};

// Pairs are read kBatch times 64 at a time, so that their latencies overlap: a lane's experts of
// the pairs p + lane, p + 64 + lane, ..., -1 where there is none
constexpr int kBatch = 4;
__device__ __forceinline__ void load_batch(const PlaceArgs &a, int64_t p, int64_t p1, int (&e)[kBatch]) {
    const int64_t i = p + (threadIdx.x & 63);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) e[u] = i + 64 * u < p1 ? a.experts[i + 64 * u] - a.first : -1;
}
__device__ __forceinline__ void count_batch(const PlaceArgs &a, const int (&e)[kBatch], uint32_t *hist) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
        if ((uint32_t)e[u] < (uint32_t)a.E) atomicAdd(&hist[e[u]], 1u);
}

__global__ __launch_bounds__(PT) void place_count_kernel(PlaceArgs a) {
    __shared__ uint32_t hist[kMaxExperts];
    const int wave = threadIdx.x >> 6;
    const int64_t p0 = ((int64_t)blockIdx.x * PW + wave) * a.seg, p1 = min(p0 + a.seg, a.pairs);
    int e[kBatch];
    load_batch(a, p0, p1, e);
    for (int x = threadIdx.x; x < a.E; x += PT) hist[x] = 0;
    __syncthreads();
    for (int64_t p = p0; p < p1; p += 64 * kBatch) {
        if (p != p0) load_batch(a, p, p1, e);
        count_batch(a, e, hist);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += PT) a.counts[(int64_t)blockIdx.x * a.E + e] = hist[e];
}

// exclusive prefix over the workgroup's threads; *all: the total
__device__ __forceinline__ uint32_t prefix(uint32_t v, uint32_t *scratch, uint32_t *all) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t s = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t o = __shfl_up(s, d, 64);
        s += lane >= d ? o : 0u;
    }
    if (lane == 63) scratch[wave] = s;
    __syncthreads();
    uint32_t before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < PW; ++w) {
        before += w < wave ? scratch[w] : 0u;
        total += scratch[w];
    }
    *all = total;
    return before + s - v;
}

__global__ __launch_bounds__(PT) void place_kernel(PlaceArgs a) {
    __shared__ uint32_t hist[PW][kMaxExperts];
    __shared__ uint32_t total[kMaxExperts], before[kMaxExperts];   // several chunks: of all, of the earlier ones
    __shared__ uint32_t scratch[PW];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t p0 = ((int64_t)blockIdx.x * PW + wave) * a.seg, p1 = min(p0 + a.seg, a.pairs);
    int batch[kBatch];
    load_batch(a, p0, p1, batch);
    for (int e = threadIdx.x; e < a.E; e += PT) {
#pragma unroll
        for (int w = 0; w < PW; ++w) hist[w][e] = 0;
        total[e] = before[e] = 0;
    }
    __syncthreads();
    if (a.chunks > 1) {
        // the columns of the table [chunks][E], a column's chunks dealt to several threads, 8 loads in
        // flight; sums of integers, whose order does not matter
        const int width = min(a.E, PT), split = PT / width, part = threadIdx.x / width;
        for (int e = threadIdx.x - part * width; e < a.E && part < split; e += width) {
            uint32_t sum = 0, earlier = 0;
            for (int c0 = part; c0 < a.chunks; c0 += 8 * split) {
                uint32_t n[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const int c = c0 + u * split;
                    n[u] = c < a.chunks ? a.counts[(int64_t)c * a.E + e] : 0u;
                }
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    sum += n[u];
                    earlier += c0 + u * split < (int)blockIdx.x ? n[u] : 0u;
                }
            }
            atomicAdd(&total[e], sum);
            atomicAdd(&before[e], earlier);
        }
    }
    for (int64_t p = p0; p < p1; p += 64 * kBatch) {
        if (p != p0) load_batch(a, p, p1, batch);
        count_batch(a, batch, hist[wave]);
    }
    __syncthreads();

    constexpr int PER = kMaxExperts / PT;   // experts of a thread
    uint32_t mine[PER], sum = 0;
#pragma unroll
    for (int u = 0; u < PER; ++u) {
        const int e = threadIdx.x * PER + u;
        mine[u] = 0;
        if (e < a.E) {
            uint32_t here = 0;
#pragma unroll
            for (int w = 0; w < PW; ++w) {
                const uint32_t c = hist[w][e];
                hist[w][e] = here;
                here += c;
            }
            mine[u] = a.chunks == 1 ? here : total[e];
        }
        sum += mine[u];
    }
    uint32_t all;
    uint32_t at = prefix(sum, scratch, &all);
#pragma unroll
    for (int u = 0; u < PER; ++u) {
        const int e = threadIdx.x * PER + u;
        if (e < a.E) {
            const uint32_t first = at + before[e];
#pragma unroll
            for (int w = 0; w < PW; ++w) hist[w][e] += first;
            if (blockIdx.x == 0) a.offsets[e] = at;
        }
        at += mine[u];
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) a.offsets[a.E] = all;
    // rows that no pair fills
    for (int64_t r = all + (int64_t)blockIdx.x * PT + threadIdx.x; r < a.pairs; r += (int64_t)a.chunks * PT)
        a.rows[r] = -1;
    __syncthreads();

    uint32_t *next = hist[wave];
    const int bits = 32 - __builtin_clz(a.E);
    for (int64_t p = p0; p < p1; p += 64 * kBatch) {
        if (p1 - p0 > 64 * kBatch) load_batch(a, p, p1, batch);   // (otherwise they are still there)
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (p + 64 * u >= p1) break;
            const int64_t i = p + 64 * u + lane;
            const int e = batch[u];
            const bool there = (uint32_t)e < (uint32_t)a.E;
            const uint64_t placed = __ballot(there);
            uint32_t lo = (uint32_t)placed, hi = (uint32_t)(placed >> 32);   // the lanes with this lane's expert
            for (int b = 0; b < bits; ++b) {
                const uint32_t bit = (uint32_t)__builtin_amdgcn_sbfe(e, b, 1);   // 0 or all ones
                const uint64_t set = __ballot(bit != 0);
                lo &= ~((uint32_t)set ^ bit);
                hi &= ~((uint32_t)(set >> 32) ^ bit);
            }
            if (there) {
                const uint32_t r = next[e] + __builtin_amdgcn_mbcnt_hi(hi, __builtin_amdgcn_mbcnt_lo(lo, 0u));
                a.slots[i] = (int32_t)r;
                a.rows[r] = (int32_t)((uint32_t)i / (uint32_t)a.k);
                // (LDS accesses of a wave run in order; the fence keeps the compiler's order)
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                const uint64_t same = ((uint64_t)hi << 32) | lo;
                if ((same >> lane) == 1ull) next[e] = r + 1;   // the last of these lanes
            } else if (i < p1) {
                a.slots[i] = -1;
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
    }
}

// Where there are several chunks, each of their workgroups reads the whole table of counts, and
// its waves walk their pairs one after another: the time is some a * chunks * E + b * pairs /
// chunks, least at chunks = sqrt(b pairs / (a E)). Measured best, us: 131072 pairs of 256 experts 10.0 at
// 64 chunks (32: 10.1, 128: 11.7), of 32 experts 7.2 at 128 (32: 8.5), of 1024 experts 15.0 at 32 (64: 18.2,
// 128: 27); 524288 pairs of 256 experts 15.0 at 128 (64: 16.6, 256: 19).
int64_t chunks_of(int64_t pairs, int64_t E) {
    if (pairs <= kOneChunk) return 1;
    const int64_t most = (pairs + kChunk - 1) / kChunk, best = (int64_t)std::sqrt(6.0 * (double)pairs / (double)E);
    const int64_t c = best < most ? best : most;
    return c < 2 ? 2 : (c < kMaxChunks ? c : kMaxChunks);
}

// ---------------------------------------------------------------------------------------

struct CombineArgs {
    const void *h;
    const int32_t *slots;
    const float *weights;   // or null: every weight 1
    void *y;
    const void *dy;
    void *dh;
    float *dweights;
    int64_t T, H, rows;
    int k;
};

// 16 bytes at any element's address: rows of any length and alignment are read and written so
// (6958 x 3 x 1447 bf16 17 us, element by element 43)
typedef u32x4 __attribute__((aligned(2))) u32x4_any;

template <int STREAM>
__device__ __forceinline__ u32x4 load16(const void *p) {
    if constexpr (STREAM) return __builtin_nontemporal_load(reinterpret_cast<const u32x4_any *>(p));
    else return *reinterpret_cast<const u32x4_any *>(p);
}

// VEC = 16 bytes of consecutive elements, BF16 or fp32. Whole pieces are stored past the caches:
// nothing here reads them again, and what the caches hold of the inputs stays (the gradient of
// 2047 x 6 x 7168 80 -> 60 us). STREAM loads them past the caches too. Of a piece of fewer than VEC
// elements (a row shorter than that) the first n count.
template <int BF16>
struct Piece {
    static constexpr int VEC = BF16 ? 8 : 4;
    float v[VEC];
    template <int STREAM = 0>
    __device__ __forceinline__ void load(const void *p, int64_t i) {
        set(load16<STREAM>(reinterpret_cast<const uint8_t *>(p) + i * (BF16 ? 2 : 4)));
    }
    __device__ __forceinline__ void store(void *p, int64_t i) const {
        __builtin_nontemporal_store(get(), reinterpret_cast<u32x4_any *>(reinterpret_cast<uint8_t *>(p) + i * (BF16 ? 2 : 4)));
    }
    __device__ __forceinline__ void load_some(const void *p, int64_t i, int n) {
        u32x4 u = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            if (j >= n) continue;
            if constexpr (BF16) u[j / 2] |= (uint32_t) reinterpret_cast<const uint16_t *>(p)[i + j] << (16 * (j & 1));
            else u[j] = reinterpret_cast<const uint32_t *>(p)[i + j];
        }
        set(u);
    }
    __device__ __forceinline__ void store_some(void *p, int64_t i, int n) const {
        const u32x4 u = get();
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            if (j >= n) continue;
            if constexpr (BF16) reinterpret_cast<uint16_t *>(p)[i + j] = (uint16_t)(u[j / 2] >> (16 * (j & 1)));
            else reinterpret_cast<uint32_t *>(p)[i + j] = u[j];
        }
    }
    __device__ __forceinline__ void set(const u32x4 &u) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            if constexpr (BF16) v[j] = j & 1 ? bf16hi_to_f32(u[j / 2]) : bf16lo_to_f32(u[j / 2]);
            else v[j] = __uint_as_float(u[j]);
        }
    }
    __device__ __forceinline__ u32x4 get() const {
        u32x4 u;
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            if constexpr (BF16) u[d] = pack_bf16x2(v[2 * d], v[2 * d + 1]);
            else u[d] = __float_as_uint(v[d]);
        }
        return u;
    }
};

// Where a row's pieces lie. WHOLE: its length is a multiple of VEC. Otherwise the last piece is the
// row's last VEC elements, the first `again` of which belong to the piece before as well (both
// write the same values there); and a row of fewer than VEC elements is one piece of n.
template <int VEC, int WHOLE>
struct Place {
    int64_t col;
    int again, n;
    __device__ __forceinline__ Place(int64_t piece, int64_t H) : col(piece * VEC), again(0), n(VEC) {
        if constexpr (!WHOLE) {
            if (H < VEC) {
                n = (int)H;
            } else if (col + VEC > H) {
                again = (int)(col + VEC - H);
                col -= again;
            }
        }
    }
};
// all but rows shorter than a piece
template <int VEC, int WHOLE>
__device__ __forceinline__ bool long_row(int64_t H) {
    return WHOLE || H >= VEC;
}

constexpr int KB = 8;     // choices whose rows are in flight together
constexpr int CT = 128;   // threads of a combine workgroup

// A workgroup sums a piece of one token's row. STREAM, for more rows than the 256 MB behind the
// L2s can hold: loaded past the caches, the pieces of a row by neighbouring workgroups (whole
// 14 KB rows at a time from memory): 8192 x 8 x 7168 bf16 213 -> 174 us, 6.1 TB/s. Rows that an
// expert's product has just left there are read with ordinary loads, a token's pieces far apart:
// 2047 x 6 x 7168 30 us, against 36 the other way.
template <int BF16, int STREAM, int WHOLE>
__global__ __launch_bounds__(CT) void combine_kernel(CombineArgs a) {
    constexpr int VEC = Piece<BF16>::VEC;
    int64_t t = blockIdx.x, piece = blockIdx.y;
    if constexpr (STREAM) {
        const int64_t n = (a.H + CT * VEC - 1) / (CT * VEC);
        piece = blockIdx.x % n;
        t = blockIdx.x / n;
    }
    piece = piece * CT + threadIdx.x;
    if (piece * VEC >= a.H) return;
    const Place<VEC, WHOLE> at(piece, a.H);
    const bool whole = long_row<VEC, WHOLE>(a.H);
    float acc[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc[i] = 0.0f;
    for (int j0 = 0; j0 < a.k; j0 += KB) {
        Piece<BF16> p[KB];
        float w[KB];
#pragma unroll
        for (int u = 0; u < KB; ++u) {
            const int j = j0 + u;
            const int s = j < a.k ? a.slots[t * a.k + j] : -1;
            w[u] = 0.0f;
#pragma unroll
            for (int i = 0; i < VEC; ++i) p[u].v[i] = 0.0f;
            if (s >= 0 && s < a.rows) {
                w[u] = a.weights ? a.weights[t * a.k + j] : 1.0f;
                if (whole) p[u].template load<STREAM>(a.h, (int64_t)s * a.H + at.col);
                else p[u].load_some(a.h, (int64_t)s * a.H, at.n);
            }
        }
#pragma unroll
        for (int u = 0; u < KB; ++u)
#pragma unroll
            for (int i = 0; i < VEC; ++i) acc[i] = __builtin_fmaf(w[u], p[u].v[i], acc[i]);
    }
    Piece<BF16> out;
#pragma unroll
    for (int i = 0; i < VEC; ++i) out.v[i] = acc[i];
    if (whole) out.store(a.y, t * a.H + at.col);
    else out.store_some(a.y, t * a.H, at.n);
}

// dh[slot] = w dy and dw = <dy, h[slot]>, a workgroup per token: each row of h is read and
// each row of dh written once. The dot products are summed in fp32 in a fixed order.
// THREADS: as many as keep all tokens on the GPU at once (its registers allow 1024 threads a CU): 512
// up to 256 tokens (64 x 8 x 7168 11 -> 9 us), 256 up to 1024, else 128 (2047 x 6 x 7168 84 -> 73 us with
// STREAM, 5.2 TB/s).
template <int BF16, int THREADS, int STREAM, int WHOLE>
__global__ __launch_bounds__(THREADS) void combine_grad_kernel(CombineArgs a) {
    constexpr int VEC = Piece<BF16>::VEC;
    __shared__ float part[THREADS / 64][KB];
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const bool whole = long_row<VEC, WHOLE>(a.H);
    for (int j0 = 0; j0 < a.k; j0 += KB) {
        int slot[KB];
        float w[KB], dot[KB];
#pragma unroll
        for (int u = 0; u < KB; ++u) {
            const int j = j0 + u;
            const int s = j < a.k ? a.slots[t * a.k + j] : -1;
            slot[u] = s < a.rows ? s : -1;
            w[u] = slot[u] >= 0 ? a.weights[t * a.k + j] : 0.0f;
            dot[u] = 0.0f;
        }
        for (int64_t piece = threadIdx.x; piece * VEC < a.H; piece += THREADS) {
            const Place<VEC, WHOLE> at(piece, a.H);
            Piece<BF16> g, p[KB], out;
            if (whole) g.load(a.dy, t * a.H + at.col);
            else g.load_some(a.dy, t * a.H, at.n);
#pragma unroll
            for (int u = 0; u < KB; ++u) {
                if (slot[u] >= 0) {
                    if (whole) p[u].template load<STREAM>(a.h, (int64_t)slot[u] * a.H + at.col);
                    else p[u].load_some(a.h, (int64_t)slot[u] * a.H, at.n);
                }
            }
#pragma unroll
            for (int u = 0; u < KB; ++u) {
                if (slot[u] >= 0) {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        // counted once: neither factor of the other time, either may be infinite
                        const bool once = WHOLE || i >= at.again;
                        dot[u] = __builtin_fmaf(once ? g.v[i] : 0.0f, once ? p[u].v[i] : 0.0f, dot[u]);
                        out.v[i] = w[u] * g.v[i];
                    }
                    if (whole) out.store(a.dh, (int64_t)slot[u] * a.H + at.col);
                    else out.store_some(a.dh, (int64_t)slot[u] * a.H, at.n);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < KB; ++u) {
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) dot[u] += __shfl_xor(dot[u], m, 64);
            if (lane == 0) part[wave][u] = dot[u];
        }
        __syncthreads();
        if (threadIdx.x < KB && j0 + (int)threadIdx.x < a.k) {
            float sum = 0.0f;
#pragma unroll
            for (int v = 0; v < THREADS / 64; ++v) sum += part[v][threadIdx.x];
            a.dweights[t * a.k + j0 + threadIdx.x] = sum;
        }
        __syncthreads();
    }
}

}  // namespace

size_t moe_place_workspace_bytes(int64_t pairs, int64_t E) {
    const int64_t c = chunks_of(pairs, E);
    return c == 1 ? 0 : (size_t)(c * E * 4);
}

hipError_t launch_moe_place(const int32_t *experts, int64_t *offsets, int32_t *rows, int32_t *slots, int64_t T, int k,
                            int E, int first, void *workspace, hipStream_t stream) {
    PlaceArgs a{experts, offsets, rows, slots, static_cast<uint32_t *>(workspace), T * k, 0, E, first, k, 0};
    a.chunks = (int)chunks_of(a.pairs, E);
    const int64_t waves = (int64_t)a.chunks * PW;
    a.seg = ((a.pairs + waves - 1) / waves + 63) / 64 * 64;
    if (a.chunks > 1) {
        place_count_kernel<<<dim3(a.chunks), dim3(PT), 0, stream>>>(a);
        if (hipError_t e = hipGetLastError()) return e;
    }
    place_kernel<<<dim3(a.chunks), dim3(PT), 0, stream>>>(a);
    return hipGetLastError();
}

template <int BF16, int WHOLE>
void combine(const CombineArgs &a, hipStream_t stream) {
    constexpr int VEC = Piece<BF16>::VEC;
    const int64_t per = CT * VEC, pieces = (a.H + per - 1) / per;
    const bool stream_rows = a.T * a.k * a.H * (16 / VEC) > ((int64_t)256 << 20) && a.T * pieces * CT <= 0xFFFFFFFFll;
    if (stream_rows)
        combine_kernel<BF16, 1, WHOLE><<<dim3((unsigned)(a.T * pieces)), dim3(CT), 0, stream>>>(a);
    else
        combine_kernel<BF16, 0, WHOLE><<<dim3((unsigned)a.T, (unsigned)pieces), dim3(CT), 0, stream>>>(a);
}

template <int BF16, int WHOLE>
void combine_grad(const CombineArgs &a, hipStream_t stream) {
    const dim3 grid((unsigned)a.T);
    // (h and dh past what the caches hold: the forward pass's h is no longer there)
    const bool stream_rows = a.T > 1024 && a.T * a.k * a.H * (16 / Piece<BF16>::VEC) > ((int64_t)128 << 20);
    if (stream_rows) combine_grad_kernel<BF16, 128, 1, WHOLE><<<grid, dim3(128), 0, stream>>>(a);
    else if (a.T <= 256) combine_grad_kernel<BF16, 512, 0, WHOLE><<<grid, dim3(512), 0, stream>>>(a);
    else if (a.T <= 1024) combine_grad_kernel<BF16, 256, 0, WHOLE><<<grid, dim3(256), 0, stream>>>(a);
    else combine_grad_kernel<BF16, 128, 0, WHOLE><<<grid, dim3(128), 0, stream>>>(a);
}

hipError_t launch_moe_combine(const void *h, bool bf16, const int32_t *slots, const float *weights, void *y, int64_t T,
                              int64_t rows, int64_t H, int k, hipStream_t stream) {
    const CombineArgs a{h, slots, weights, y, nullptr, nullptr, nullptr, T, H, rows, k};
    if (bf16) H % 8 ? combine<1, 0>(a, stream) : combine<1, 1>(a, stream);
    else H % 4 ? combine<0, 0>(a, stream) : combine<0, 1>(a, stream);
    return hipGetLastError();
}

hipError_t launch_moe_combine_backward(const void *dy, const void *h, bool bf16, const int32_t *slots,
                                       const float *weights, void *dh, float *dweights, int64_t T, int64_t rows,
                                       int64_t H, int k, hipStream_t stream) {
    const CombineArgs a{h, slots, weights, nullptr, dy, dh, dweights, T, H, rows, k};
    if (bf16) H % 8 ? combine_grad<1, 0>(a, stream) : combine_grad<1, 1>(a, stream);
    else H % 4 ? combine_grad<0, 0>(a, stream) : combine_grad<0, 1>(a, stream);
    return hipGetLastError();
}

}  // namespace fp8q
