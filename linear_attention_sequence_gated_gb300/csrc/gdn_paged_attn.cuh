// Decode attention over a paged cache of 16- or 32-bit rows (gdn_flash_attn_paged): for
// every sequence b, query head h and query i,
//     out[b, i, h, :] = softmax_j(scale q[b,h,i] . k[b,hk,j] + mask[b,0,i,j]) v[b,hk,j,:]
// over the tokens j that the sequence holds (with `causal`, up to the query's own), hk = h /
// (n_heads / n_heads_kv), row j of sequence b in page table[b][j / page] at j % page.
//
// The cache is streamed once: (dk + dv) e bytes a token and kv head against 2 (dk + dv) flops
// a row = (query head of the group, query), so up to some 25 rows HBM bounds the call and the
// kernel's work is to keep copies in flight.
//   * A tile is 16 tokens of one kv head, which never leave a page.  A warp streams tiles through
//     a ring of its own in shared memory, filled by TMA boxes of 16 tokens x 128 bytes with
//     128-byte swizzling (any order of a cache's tokens and heads: the tensor map holds the
//     strides), whose rows ldmatrix reads without bank conflicts.
//   * 16-bit rows: S^T = K Q^T (M = 16 tokens, N = 8 rows) and O^T += V^T P^T (M = 16 elements,
//     N = 8 rows, K = 16 tokens) by m16n8k16 MMAs with fp32 accumulators; the weights as hi + lo
//     16-bit pairs (16 bits of bf16, 22 of f16), transposed in registers by movmatrix.
//   * fp32 rows: the same by m16n8k8 tf32 MMAs, each operand as hi + lo (22 bits), three products.
//   * Scores, maxima, sums and outputs are fp32; each tile's products reach the outputs by one
//     fp32 FMA, since the MMAs' own accumulation truncates.
//
// Work is shared out in tiles, not in sequences: the tiles of all units (sequence, kv head, block
// of rows) in a row are cut into equal runs, one a CTA, so ragged batches and single long
// sequences load the GPU evenly.  The warps of a CTA take the tiles of a unit in turn and join
// their parts in shared memory at its end, while the next unit's copies are in flight.  A unit
// that runs cut leaves (max, sum, output) in the workspace, and a second kernel joins those parts
// in a fixed order.  A call of few tiles gives each unit a cluster of CTAs instead, which join
// through distributed shared memory: one launch, no workspace.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <type_traits>

#include "../../include/gdn.h"
#include "gdn_internal.h"
#include "gdn_kv4.cuh"
#include "gdn_ptx.cuh"

namespace gdn {
namespace paged {

constexpr int kTile = 16;              // tokens of a tile
constexpr int kBlock = 8;              // rows of an MMA column tile
constexpr int kGrid = 152;             // runs at most: one CTA per SM of the GPU this is written for (the
                                       // workspace's size goes by it on any device)
constexpr int kMaxCluster = 8;         // the largest portable size

struct Attn {
    const void *q, *mask;
    void *out;
    float *ws;
    const int *table, *lens;
    int *status;
    long long q_seq, q_head, q_query;  // in elements
    int n_seqs, H, Hkv, n_q, R, n_rb;  // R rows a kv head in n_rb blocks
    int n_pages, tpp, max_pages;       // tpp: tiles of a page
    float scale;
    int out_type, cluster;             // CTAs a unit, or 0: equal runs
    bool causal;
    int k_order, v_order;              // of the tensor maps' outer coordinates: two bits each, 0 token, 1 head, 2 page
};

// Blocks of 8 rows that a unit takes: the cache is read once for all of them.  (Four of them fill the
// registers where a width is 256.)
constexpr int blocks_of(bool wide, bool fp32, int R) {
    return fp32 || R <= kBlock ? 1 : R <= 2 * kBlock || wide ? 2 : 4;
}
// Warps of a CTA: 8 with tiles of 8 KB, fewer with larger ones, so that the ring holds 2 or 3 a warp.
constexpr int warps_of(int dk, int dv, int elt) {
    return kTile * (dk + dv) * elt <= 8192 ? 8 : kTile * (dk + dv) * elt <= 16384 ? 4 : 2;
}

// The kernel for rows of type T and keys of width DK (one translation unit each).
template <typename T, int DK>
cudaError_t launch_attn(int dv, const CUtensorMap &km, const CUtensorMap &vm, const Attn &a, int grid,
                        cudaStream_t stream);

#ifdef GDN_PAGED_ATTN_T
namespace {

using kv4::run_begin;
using kv4::run_of;
using kv4::partial_slot;

constexpr int kSmemMax = 227 * 1024;

// Shape of the kernel for widths DK and DV, type T and NB blocks of 8 rows.
template <typename T, int DK, int DV, int NB>
struct Geo {
    static constexpr int E = (int)sizeof(T);
    static constexpr bool MMA16 = E == 2;
    static constexpr int BOX = 128 / E;                // elements of a box's row
    static constexpr int KB = kTile * DK * E, VB = kTile * DV * E, STAGE = KB + VB;
    static constexpr int WARPS = warps_of(DK, DV, E);
    static constexpr int THREADS = WARPS * 32;
    static constexpr int ROWS = NB * kBlock;
    // the warps' outputs of 8 rows, to be joined
    static constexpr int MERGE = WARPS * kBlock * DV * 4;
    // queries in shared memory, rows padded against bank conflicts: 16-bit ones (one block stays in registers), fp32
    // ones as hi and lo
    static constexpr int QROW = MMA16 ? DK * 2 + 16 : DK * 8 + 64;
    static constexpr int Q = MMA16 && NB == 1 ? 0 : ROWS * QROW;
    static constexpr int PT = MMA16 ? 0 : WARPS * kBlock * 20 * 4;     // fp32 weights on their way to B operands
    static constexpr int ML = 2 * (WARPS + 1) * ROWS * 4;
    static constexpr int FIXED = 1024 + MERGE + Q + PT + ML;               // (1024: the ring's alignment)
    static constexpr int FIT = (kSmemMax - 768 - FIXED) / (WARPS * STAGE);  // (768: barriers and the like)
    static constexpr int STAGES = FIT < 6 ? FIT : 6;
    static constexpr int RING = WARPS * STAGES * STAGE;
    static constexpr int SMEM = RING + FIXED;
    static_assert(STAGES >= 2, "ring");
    static_assert(MERGE % 16 == 0 && Q % 16 == 0 && PT % 16 == 0 && ML % 8 == 0, "alignment");
};

constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 2^((a - b) log2 e), 0 for a = -inf, whatever b
__device__ __forceinline__ float weight(float a, float b) {
    return a == -INFINITY ? 0.f : exp2_approx((a - b) * kLog2e);
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
    uint4 x;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(a) : "memory");
    return x;
}
template <typename T>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
            "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else if constexpr (std::is_same<T, __half>::value)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
            "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 "
            "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 8 x 8 transpose of 16-bit elements across the warp: lane (g, t) gives row g, columns 2t,
// 2t + 1 and gets row g of the transpose.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// (x, y) as 16-bit pairs hi + lo
template <typename T>
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        const float2 f = __bfloat1622float2(h);
        const __nv_bfloat162 l = __floats2bfloat162_rn(x - f.x, y - f.y);
        hi = *reinterpret_cast<const uint32_t *>(&h);
        lo = *reinterpret_cast<const uint32_t *>(&l);
    } else {
        const __half2 h = __floats2half2_rn(x, y);
        const float2 f = __half22float2(h);
        const __half2 l = __floats2half2_rn(x - f.x, y - f.y);
        hi = *reinterpret_cast<const uint32_t *>(&h);
        lo = *reinterpret_cast<const uint32_t *>(&l);
    }
}
// fp32 as tf32 hi + lo: 11 bits each, to nearest, so 22 of the value's 24
__device__ __forceinline__ void split_tf32(float x, uint32_t &hi, uint32_t &lo) {
    hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
    const float r = x - __uint_as_float(hi);
    lo = (__float_as_uint(r) + 0x1000u) & 0xffffe000u;
    if (r != r) lo = 0x7fffffffu;      // (a NaN's payload may carry into the sign; an infinity is NaN too)
}

template <typename T> __device__ __forceinline__ float to_float(T x);
template <> __device__ __forceinline__ float to_float<float>(float x) { return x; }
template <> __device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <> __device__ __forceinline__ float to_float<__half>(__half x) { return __half2float(x); }

// 4 consecutive outputs
__device__ __forceinline__ void store4(void *out, int type, size_t i, float4 x) {
    if (type == GDN_DTYPE_F32) {
        *reinterpret_cast<float4 *>(static_cast<float *>(out) + i) = x;
        return;
    }
    uint2 w;
    if (type == GDN_DTYPE_BF16) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
        w = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    } else {
        const __half2 a = __floats2half2_rn(x.x, x.y), b = __floats2half2_rn(x.z, x.w);
        w = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    }
    *reinterpret_cast<uint2 *>(static_cast<unsigned short *>(out) + i) = w;
}

__device__ __forceinline__ int capacity(const Attn &a) { return a.max_pages * a.tpp * kTile; }
__device__ __forceinline__ int tiles_at(const Attn &a, int b) {
    return (min(max(a.lens[b], 0), capacity(a)) + kTile - 1) / kTile;
}
__device__ __forceinline__ int units_of(const Attn &a) { return a.Hkv * a.n_rb; }     // of a sequence

// A partial result: [rows][DV] outputs, [rows] maxima, [rows] sums.
template <int ROWS, int DV> constexpr size_t kPartial = (size_t)ROWS * (DV + 2);

// Sum of x over the block, in every thread; `part` is 32 ints, free again after the next barrier.
__device__ __forceinline__ int block_sum(int x, int *part, int warps) {
    x = __reduce_add_sync(0xffffffffu, x);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    return __reduce_add_sync(0xffffffffu, lane < warps ? part[lane] : 0);
}

// Tiles of all units; a length beyond the table shows in the status word.
__device__ __forceinline__ int total_tiles(const Attn &a, int *part, int threads) {
    int n = 0;
    for (int b = threadIdx.x; b < a.n_seqs; b += threads) {
        n += tiles_at(a, b);
        if (a.lens[b] > capacity(a)) *a.status = GDN_ERR_PAGE;
    }
    return block_sum(n, part, threads / 32) * units_of(a);
}

// Whole warp: the sequence that tile x of all lies in, and the tiles before it.
__device__ __forceinline__ int find_tile(const Attn &a, int x, int lane, int *before) {
    int done = 0;
    for (int base = 0;; base += 32) {
        const int n = base + lane < a.n_seqs ? tiles_at(a, base + lane) * units_of(a) : 0;
        int incl = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += o;
        }
        incl += done;
        const unsigned hit = __ballot_sync(0xffffffffu, incl > x);
        if (hit || base + 32 >= a.n_seqs) {            // (x is below the total, so there is one)
            const int src = hit ? __ffs(hit) - 1 : 31;
            *before = __shfl_sync(0xffffffffu, incl - n, src);
            return min(base + src, a.n_seqs - 1);
        }
        done = __shfl_sync(0xffffffffu, incl, 31);
    }
}

// Runs of a call of T tiles: fewer where they would have less than a tile for each warp.
__device__ __forceinline__ int runs_of(int T, int warps) { return min(kGrid, (T + warps - 1) / warps); }

// A walk over the tiles of a CTA's run: a segment is the part of a unit that lies in it.
struct Walk {
    int left;                          // tiles of the run from this segment on
    int b, j;                          // sequence, unit in it
    int begin, end, n;                 // tiles [begin, end) of the unit's n
    __device__ __forceinline__ void cut() { end = min(n, begin + left); }
    __device__ __forceinline__ bool next(const Attn &a) {
        left -= end - begin;
        if (left <= 0) return false;
        begin = 0;
        if (++j == units_of(a)) {
            j = 0;
            do {
                if (++b >= a.n_seqs) return false;
                n = tiles_at(a, b);
            } while (n == 0);
        }
        cut();
        return true;
    }
};

// What fills a warp's ring: a walk that runs ahead of the computation.
template <typename G>
struct Feed {
    Walk w;
    bool more;
    int at;                            // the warp's next tile of the segment
    int page, off;                     // lane i: page and first token in it of its tile first + i * WARPS
    int first;
    uint32_t bad;                      // stages whose tile is in no page of the cache

    __device__ __forceinline__ void look(const Attn &a, int lane) {
        first = at;
        const int tile = at + lane * G::WARPS;
        page = -1;
        off = 0;
        if (more && tile < w.end) {
            const int slot = tile / a.tpp;
            page = a.table[(size_t)w.b * a.max_pages + slot];
            off = (tile - slot * a.tpp) * kTile;
        }
    }
    __device__ __forceinline__ void start(const Attn &a, const Walk &run, bool any, int warp, int lane) {
        w = run;
        more = any;
        bad = 0;
        at = w.begin + warp;
        settle(a, warp);
        look(a, lane);
    }
    // on to a segment in which this warp has a tile
    __device__ __forceinline__ bool settle(const Attn &a, int warp) {
        bool moved = false;
        while (more && at >= w.end) {
            more = w.next(a);
            at = w.begin + warp;
            moved = true;
        }
        return moved;
    }
    __device__ __forceinline__ void issue(const Attn &a, const CUtensorMap *km, const CUtensorMap *vm, uint8_t *stage,
                                          uint64_t *bar, int s, int warp, int lane) {
        if (!more) return;
        const int i = (at - first) / G::WARPS;
        const int p = __shfl_sync(0xffffffffu, page, i), o = __shfl_sync(0xffffffffu, off, i);
        const bool ok = (unsigned)p < (unsigned)a.n_pages;
        bad = ok ? bad & ~(1u << s) : bad | 1u << s;
        if (lane == 0) {
            if (!ok) {
                *a.status = GDN_ERR_PAGE;
                ptx::mbar_arrive(bar);
            } else {
                ptx::mbar_arrive_expect_tx(bar, G::STAGE);
                const int h = w.j / a.n_rb;
                auto pick = [&](int order) { return (order & 3) == 0 ? o : (order & 3) == 1 ? h : p; };
                const int k1 = pick(a.k_order), k2 = pick(a.k_order >> 2), k3 = pick(a.k_order >> 4);
                const int v1 = pick(a.v_order), v2 = pick(a.v_order >> 2), v3 = pick(a.v_order >> 4);
#pragma unroll
                for (int c = 0; c < G::KB / 2048; ++c)
                    ptx::tma_load_4d(stage + c * 2048, km, bar, c * G::BOX, k1, k2, k3);
#pragma unroll
                for (int c = 0; c < G::VB / 2048; ++c)
                    ptx::tma_load_4d(stage + G::KB + c * 2048, vm, bar, c * G::BOX, v1, v2, v3);
            }
        }
        at += G::WARPS;
        if (settle(a, warp) || i == 31) look(a, lane);
    }
};

// One warp's share of one unit: an online softmax over tiles.
template <typename T, int DK, int DV, int NB, bool COLS>
struct Unit {
    using G = Geo<T, DK, DV, NB>;
    static constexpr bool MMA16 = G::MMA16;
    static constexpr int KS = DK / 16, MT = DV / 16;   // 16-element steps of a key, blocks of a value row
    // weights of f16 rows are scaled by 2^12, so that small ones keep their bits
    static constexpr float kBits = std::is_same<T, __half>::value ? 12.f : 0.f;

    uint32_t qf[MMA16 && NB == 1 ? KS : 1][2];
    float m[NB][2], l[NB][2];          // of rows 2t, 2t + 1: running maximum, this lane's sum of weights
    float o[NB][MT][4];
    int qi[NB][2];                     // the row's query; -1: no such row
    int raw, all, len;                 // length; tokens that every row sees and no mask changes; in the table
    int b;

    __device__ __forceinline__ static int row_of(int rb, int nb, int c) {
        return COLS ? c & 3 : rb * G::ROWS + nb * kBlock + c;
    }
    __device__ __forceinline__ static const T *q_row(const Attn &a, int b, int hk, int row) {
        const int h = hk * (a.H / a.Hkv) + row / a.n_q, i = row % a.n_q;
        return static_cast<const T *>(a.q) + b * a.q_seq + h * a.q_head + i * a.q_query;
    }

    // Queries to shared memory, by the whole block (a barrier follows).
    __device__ __forceinline__ static void stage_queries(const Attn &a, int b, int hk, int rb, uint8_t *sq) {
        constexpr int PER = 16 / (int)sizeof(T);
        for (int x = threadIdx.x; x < G::ROWS * (DK / PER); x += G::THREADS) {
            const int r = x / (DK / PER), c = x - r * (DK / PER), row = rb * G::ROWS + r;
            uint4 w = make_uint4(0, 0, 0, 0);
            if (row < a.R) w = *reinterpret_cast<const uint4 *>(q_row(a, b, hk, row) + c * PER);
            if constexpr (MMA16) {
                *reinterpret_cast<uint4 *>(sq + r * G::QROW + c * 16) = w;
            } else {
                uint4 hi, lo;
                split_tf32(__uint_as_float(w.x), hi.x, lo.x);
                split_tf32(__uint_as_float(w.y), hi.y, lo.y);
                split_tf32(__uint_as_float(w.z), hi.z, lo.z);
                split_tf32(__uint_as_float(w.w), hi.w, lo.w);
                *reinterpret_cast<uint4 *>(sq + r * G::QROW + c * 16) = hi;
                *reinterpret_cast<uint4 *>(sq + r * G::QROW + DK * 4 + c * 16) = lo;
            }
        }
    }

    __device__ __forceinline__ void begin(const Attn &a, int seq, int hk, int rb, int lane) {
        const int g = lane >> 2, t = lane & 3;
        b = seq;
        raw = max(a.lens[b], 0);
        len = min(raw, capacity(a));
        all = a.mask ? 0 : a.causal ? min(len, max(raw - a.n_q + 1, 0)) : len;
        if constexpr (MMA16 && NB == 1) {
            const int row = row_of(rb, 0, g);
            const bool ok = row < a.R;
            const uint32_t *p = reinterpret_cast<const uint32_t *>(q_row(a, b, hk, ok ? row : 0));
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                qf[s][0] = ok ? p[s * 8 + t] : 0u;
                qf[s][1] = ok ? p[s * 8 + 4 + t] : 0u;
            }
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = row_of(rb, nb, 2 * t + r);
                qi[nb][r] = row < a.R ? row % a.n_q : -1;
                m[nb][r] = -INFINITY;
                l[nb][r] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[nb][i][e] = 0.f;
        }
    }

    // S^T of a tile: entry e is token g + 8 (e >> 1) and row 2t + (e & 1) of block nb.
    __device__ __forceinline__ void scores(uint32_t k, const uint8_t *sq, int lane, float (&s)[NB][4]) const {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[nb][e] = 0.f;
        if constexpr (MMA16) {
            const uint32_t row = k + (lane & 15) * 128, x = lane & 7, half = lane >> 4;
            float s2[4] = {0.f, 0.f, 0.f, 0.f};        // a second chain of products where there is one block
#pragma unroll
            for (int c = 0; c < KS; ++c) {
                uint32_t A[4];
                ldsm4(A, row + (c >> 2) * 2048 + (((2 * (c & 3) + half) ^ x) << 4));
                if constexpr (NB == 1) {
                    if (c & 1) mma<T>(s2, A, qf[c][0], qf[c][1]);
                    else mma<T>(s[0], A, qf[c][0], qf[c][1]);
                } else {
                    // two blocks' B operands: rows (lane & 7) of block 2 p + (lane >> 4), half (lane >> 3) & 1
#pragma unroll
                    for (int p = 0; p < NB / 2; ++p) {
                        uint32_t B[4];
                        ldsm4(B, ptx::smem_u32(sq) + ((2 * p + (lane >> 4)) * kBlock + (lane & 7)) * G::QROW + c * 32 +
                                     ((lane >> 3) & 1) * 16);
                        mma<T>(s[2 * p], A, B[0], B[1]);
                        mma<T>(s[2 * p + 1], A, B[2], B[3]);
                    }
                }
            }
            if constexpr (NB == 1)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[0][e] += s2[e];
        } else {
            // Lane (g, t) has elements 4t .. 4t + 3 of each 16 of tokens g and g + 8: the first two
            // are columns t and t + 4 of one k8 product, the others of the next (the queries' likewise).
            // Odd g read the second 16 of each 32 first, so that 8 lanes read 8 different pieces.
            const uint32_t ra = k + g * 128, x = g & 7, odd = g & 1;
            const uint8_t *q = sq + g * G::QROW + t * 16;
            float s1[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
            for (int c = 0; c < DK / 32; ++c) {
                const uint32_t p0 = ra + c * 2048 + (((t + 4 * odd) ^ x) << 4);
                const uint32_t p1 = ra + c * 2048 + (((t + 4 * (odd ^ 1)) ^ x) << 4);
                const uint4 u0 = lds16(p0), u1 = lds16(p1), v0 = lds16(p0 + 1024), v1 = lds16(p1 + 1024);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint4 u = h == (int)odd ? u0 : u1, v = h == (int)odd ? v0 : v1;
                    const uint4 qh = *reinterpret_cast<const uint4 *>(q + c * 128 + h * 64);
                    const uint4 ql = *reinterpret_cast<const uint4 *>(q + DK * 4 + c * 128 + h * 64);
                    uint32_t hi[4], lo[4];
                    split_tf32(__uint_as_float(u.x), hi[0], lo[0]);
                    split_tf32(__uint_as_float(v.x), hi[1], lo[1]);
                    split_tf32(__uint_as_float(u.y), hi[2], lo[2]);
                    split_tf32(__uint_as_float(v.y), hi[3], lo[3]);
                    mma<T>(s1, lo, qh.x, qh.y);
                    mma<T>(s2, hi, ql.x, ql.y);
                    mma<T>(s[0], hi, qh.x, qh.y);
                    split_tf32(__uint_as_float(u.z), hi[0], lo[0]);
                    split_tf32(__uint_as_float(v.z), hi[1], lo[1]);
                    split_tf32(__uint_as_float(u.w), hi[2], lo[2]);
                    split_tf32(__uint_as_float(v.w), hi[3], lo[3]);
                    mma<T>(s1, lo, qh.z, qh.w);
                    mma<T>(s2, hi, ql.z, ql.w);
                    mma<T>(s[0], hi, qh.z, qh.w);
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) s[0][e] += s1[e] + s2[e];
        }
    }

    // Element of value row `tok` that o[.][i][e] sums, as the stage holds it.
    __device__ __forceinline__ static int element_of(int i, int e, int g) {
        return MMA16 ? i * 16 + g + 8 * (e >> 1) : (i >> 1) * 32 + 4 * g + 2 * (i & 1) + (e >> 1);
    }
    __device__ __forceinline__ static uint32_t value_at(int tok, int x) {
        return (uint32_t)((x / G::BOX) * 2048 + tok * 128 + ((((x % G::BOX) * G::E / 16) ^ (tok & 7)) << 4) +
                          x * G::E % 16);
    }

    // Values of tokens that some row must not see may be anything, infinities and NaN among them, and
    // a weight of 0 does not silence those in a product.  Where such a tile has any, the rows that
    // see them take them one by one, and the products take zeros for them.
    __device__ __forceinline__ void odd_values(uint8_t *v, const float (&p)[NB][4], const float (&x)[NB][4],
                                            const float (&cf)[NB][2], int lane) {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[nb][i][e] *= cf[nb][e & 1];
#pragma unroll 1
        for (int tok = 0; tok < kTile; ++tok) {
            const int src = (tok & 7) * 4 + t;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float w0 = __shfl_sync(0xffffffffu, p[nb][r], src), w1 = __shfl_sync(0xffffffffu, p[nb][r + 2], src);
                    const float x0 = __shfl_sync(0xffffffffu, x[nb][r], src), x1 = __shfl_sync(0xffffffffu, x[nb][r + 2], src);
                    const float w = tok < 8 ? w0 : w1, sc = tok < 8 ? x0 : x1;
                    if (sc == -INFINITY || (COLS && t >= 2)) continue;
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int e = r; e < 4; e += 2) {
                            const float y = to_float<T>(*reinterpret_cast<const T *>(v + value_at(tok, element_of(i, e, g))));
                            if (!isfinite(y)) o[nb][i][e] = fmaf(w, y, o[nb][i][e]);
                        }
                }
        }
        __syncwarp();
        for (int i = lane; i < kTile * DV; i += 32) {
            T *y = reinterpret_cast<T *>(v + value_at(i / DV, i % DV));
            if (!isfinite(to_float<T>(*y))) *y = T(0.f);
        }
        ptx::fence_proxy_async_smem();  // (the next copy into this stage comes after these stores)
        __syncwarp();
    }
    __device__ __forceinline__ static bool any_odd(const uint8_t *v, int lane) {
        bool bad = false;
#pragma unroll
        for (int i = 0; i < G::VB / 512; ++i) {
            const uint4 w = *reinterpret_cast<const uint4 *>(v + (i * 32 + lane) * 16);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (MMA16) {
                    constexpr uint32_t INF = std::is_same<T, __nv_bfloat16>::value ? 0x7f80u : 0x7c00u;
                    bad |= (u[e] & INF) == INF || (u[e] >> 16 & INF) == INF;
                } else {
                    bad |= (u[e] & 0x7f800000u) == 0x7f800000u;
                }
            }
        }
        return __any_sync(0xffffffffu, bad);
    }

    // The tile in `stage`, tokens pos .. pos + 15 of the sequence; `good`: it is there.
    __device__ __forceinline__ void tile(const Attn &a, uint8_t *stage, const uint8_t *sq, float *pt, int pos, bool good,
                                         int lane) {
        const int g = lane >> 2, t = lane & 3;
        if (!good) return;
        const uint32_t k = ptx::smem_u32(stage), v = k + G::KB;
        float s[NB][4], x[NB][4], cf[NB][2];
        scores(k, sq, lane, s);
        const bool plain = pos + kTile <= all;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
#pragma unroll
                for (int e = r; e < 4; e += 2) x[nb][e] = s[nb][e] * a.scale;
                if (!plain) {
                    const int i = qi[nb][r];
                    const long long lim = a.causal ? min((long long)len, (long long)raw - a.n_q + 1 + i) : len;
#pragma unroll
                    for (int e = r; e < 4; e += 2) {
                        const int j = pos + g + 8 * (e >> 1);
                        if (i < 0 || j >= lim) {
                            x[nb][e] = -INFINITY;
                        } else if (a.mask) {
                            const float add = to_float<T>(static_cast<const T *>(a.mask)[((size_t)b * a.n_q + i) * (size_t)capacity(a) + j]);
                            x[nb][e] = add == -INFINITY ? add : x[nb][e] + add;
                        }
                    }
                }
                float mx = fmaxf(x[nb][r], x[nb][r + 2]);
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                // Weights go by differences, 2^((x - maximum) log2 e), which are exact where they matter:
                // masks of the type's lowest value and scores of any size keep their order, and the factor of
                // earlier tiles is exactly 1 while the maximum stands.
                const float old = m[nb][r], mn = fmaxf(old, mx), base = mn == -INFINITY ? 0.f : mn;
                m[nb][r] = mn;
                cf[nb][r] = exp2_approx((old - base) * kLog2e);
                s[nb][r] = exp2_approx(fmaf(x[nb][r] - base, kLog2e, kBits));
                s[nb][r + 2] = exp2_approx(fmaf(x[nb][r + 2] - base, kLog2e, kBits));
                l[nb][r] = fmaf(l[nb][r], cf[nb][r], s[nb][r] + s[nb][r + 2]);
            }
        if (!plain && any_odd(stage + G::KB, lane)) {
            odd_values(stage + G::KB, s, x, cf, lane);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) cf[nb][0] = cf[nb][1] = 1.f;
        }
        if constexpr (MMA16) {
            uint32_t ph[NB][2], pl[NB][2];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t hi, lo;
                    split2<T>(s[nb][2 * h], s[nb][2 * h + 1], hi, lo);
                    if constexpr (COLS) {
                        ph[nb][h] = transpose8(t >= 2 ? lo : hi);      // columns 4 .. 7: the remainders
                    } else {
                        ph[nb][h] = transpose8(hi);
                        pl[nb][h] = transpose8(lo);
                    }
                }
            const uint32_t tok = (lane & 7) + ((lane >> 4) << 3);
            const uint32_t row = v + tok * 128, sw = lane & 7, half = (lane >> 3) & 1;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                uint32_t A[4];
                ldsm4_t(A, row + (i >> 2) * 2048 + (((2 * (i & 3) + half) ^ sw) << 4));
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    float d[4] = {0.f, 0.f, 0.f, 0.f};
                    if constexpr (!COLS) mma<T>(d, A, pl[nb][0], pl[nb][1]);   // small terms first
                    mma<T>(d, A, ph[nb][0], ph[nb][1]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[nb][i][e] = fmaf(o[nb][i][e], cf[nb][e & 1], d[e]);
                }
            }
        } else {
            // weights to [row][token]; lane (g, t) takes row g, tokens 2t, 2t + 1, 2t + 8, 2t + 9
            pt[(2 * t) * 20 + g] = s[0][0];
            pt[(2 * t + 1) * 20 + g] = s[0][1];
            pt[(2 * t) * 20 + g + 8] = s[0][2];
            pt[(2 * t + 1) * 20 + g + 8] = s[0][3];
            __syncwarp();
            uint32_t ph[4], pl[4];
            {
                const float2 u = *reinterpret_cast<const float2 *>(pt + g * 20 + 2 * t);
                const float2 w = *reinterpret_cast<const float2 *>(pt + g * 20 + 2 * t + 8);
                split_tf32(u.x, ph[0], pl[0]);
                split_tf32(u.y, ph[1], pl[1]);
                split_tf32(w.x, ph[2], pl[2]);
                split_tf32(w.y, ph[3], pl[3]);
            }
            // Lane (g, t) has elements 4g .. 4g + 3 of each 32 of those tokens: rows g and g + 8 of two M tiles.
            // Tokens 2t (and 2t + 1) of a phase's 8 lanes lie on different pieces.
#pragma unroll
            for (int c = 0; c < DV / 32; ++c) {
                uint32_t w[4][4];
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const int tok = 2 * t + (n & 1) + 8 * (n >> 1);
                    const uint4 y = lds16(v + c * 2048 + tok * 128 + ((g ^ (tok & 7)) << 4));
                    w[n][0] = y.x; w[n][1] = y.y; w[n][2] = y.z; w[n][3] = y.w;
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float d[4] = {0.f, 0.f, 0.f, 0.f};
                    uint32_t hi[2][4], lo[2][4];
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        split_tf32(__uint_as_float(w[2 * n][2 * i]), hi[n][0], lo[n][0]);
                        split_tf32(__uint_as_float(w[2 * n][2 * i + 1]), hi[n][1], lo[n][1]);
                        split_tf32(__uint_as_float(w[2 * n + 1][2 * i]), hi[n][2], lo[n][2]);
                        split_tf32(__uint_as_float(w[2 * n + 1][2 * i + 1]), hi[n][3], lo[n][3]);
                    }
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        mma<T>(d, lo[n], ph[2 * n], ph[2 * n + 1]);
                        mma<T>(d, hi[n], pl[2 * n], pl[2 * n + 1]);
                    }
#pragma unroll
                    for (int n = 0; n < 2; ++n) mma<T>(d, hi[n], ph[2 * n], ph[2 * n + 1]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[0][2 * c + i][e] = fmaf(o[0][2 * c + i][e], cf[0][e & 1], d[e]);
                }
            }
        }
    }

    // Sums over the lanes that share rows; in COLS, the remainders' columns.
    __device__ __forceinline__ void finish() {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1)
#pragma unroll
                for (int r = 0; r < 2; ++r) l[nb][r] += __shfl_xor_sync(0xffffffffu, l[nb][r], off);
            if constexpr (COLS)
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[nb][i][e] += __shfl_xor_sync(0xffffffffu, o[nb][i][e], 2);
        }
    }
};

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer_addr(const void *p, int rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(ptx::smem_u32(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ float peer_float(const void *p, int rank) {
    float x;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(peer_addr(p, rank)));
    return x;
}
__device__ __forceinline__ float4 peer_float4(const void *p, int rank) {
    float4 x;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "r"(peer_addr(p, rank)));
    return x;
}

__device__ __forceinline__ float4 fma4(float w, float4 x, float4 y) {
    return make_float4(fmaf(w, x.x, y.x), fmaf(w, x.y, y.y), fmaf(w, x.z, y.z), fmaf(w, x.w, y.w));
}

// Output row `row` of (b, hk), elements 4c .. : x / l
template <int DV>
__device__ __forceinline__ void write_out(const Attn &a, int b, int hk, int row, int c, float4 x, float l) {
    if (row >= a.R) return;
    const int h = hk * (a.H / a.Hkv) + row / a.n_q, i = row % a.n_q;
    const float f = l > 0.f || l != l ? 1.f / l : 0.f;
    store4(a.out, a.out_type, (((size_t)b * a.n_q + i) * a.H + h) * DV + 4 * c,
           make_float4(x.x * f, x.y * f, x.z * f, x.w * f));
}

template <typename T, int DK, int DV, int NB, bool COLS>
__global__ void __launch_bounds__(Geo<T, DK, DV, NB>::THREADS, 1)
attn_kernel(const __grid_constant__ CUtensorMap km, const __grid_constant__ CUtensorMap vm, const Attn a) {
    using G = Geo<T, DK, DV, NB>;
    using U = Unit<T, DK, DV, NB, COLS>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = smem_raw + (-ptx::smem_u32(smem_raw) & 1023u);
    float *merge = reinterpret_cast<float *>(ring + G::RING);              // [WARPS][8][DV]
    uint8_t *sq = ring + G::RING + G::MERGE;
    float *pts = reinterpret_cast<float *>(sq + G::Q);
    float *sm = reinterpret_cast<float *>(sq + G::Q + G::PT);              // [WARPS + 1][ROWS] maxima
    float *sl = sm + (G::WARPS + 1) * G::ROWS;                             // ... and sums; the last: the block's
    __shared__ uint64_t full[G::WARPS][G::STAGES];
    __shared__ int part[32], start[2], gave_up;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (lane == 0) {
        for (int s = 0; s < G::STAGES; ++s) ptx::mbar_init(&full[warp][s], 1);
        ptx::fence_mbar_init();
    }
    if (tid == 0) {
        gave_up = 0;
        if (a.n_pages) {
            ptx::prefetch_tmap(&km);
            ptx::prefetch_tmap(&vm);
        }
    }
    kv4::after_the_kernel_before();

    // ---- this CTA's run
    Walk run{0, 0, 0, 0, 0, 0};
    int rank = 0, cta = 0;
    if (a.cluster) {
        rank = (int)(blockIdx.x % (unsigned)a.cluster);
        const int unit = (int)(blockIdx.x / (unsigned)a.cluster);
        run.b = unit / units_of(a);
        run.j = unit - run.b * units_of(a);
        run.n = tiles_at(a, run.b);
        if (tid == 0 && a.lens[run.b] > capacity(a)) *a.status = GDN_ERR_PAGE;
        run.begin = (int)((long long)run.n * rank / a.cluster);
        run.end = (int)((long long)run.n * (rank + 1) / a.cluster);
        run.left = run.end - run.begin;
        __syncthreads();
    } else {
        cta = (int)blockIdx.x;
        const int total = total_tiles(a, part, G::THREADS);
        const int runs = runs_of(total, G::WARPS);
        const int from = cta < runs ? run_begin(total, runs, cta) : 0;
        run.left = cta < runs ? run_begin(total, runs, cta + 1) - from : 0;
        if (warp == 0 && run.left > 0) {
            int before;
            const int b = find_tile(a, from, lane, &before);
            if (lane == 0) {
                start[0] = b;
                start[1] = from - before;
            }
        }
        // rows of empty sequences
        for (int b = cta; b < a.n_seqs; b += gridDim.x)
            if (tiles_at(a, b) == 0)
                for (int i = tid; i < a.n_q * a.H * (DV / 4); i += G::THREADS)
                    store4(a.out, a.out_type, (size_t)b * a.n_q * a.H * DV + 4 * (size_t)i, make_float4(0.f, 0.f, 0.f, 0.f));
        __syncthreads();
        if (run.left > 0) {
            run.b = start[0];
            run.n = tiles_at(a, run.b);
            run.j = start[1] / run.n;
            run.begin = start[1] - run.j * run.n;
            run.cut();
        }
    }
    const bool any = run.left > 0;

    uint8_t *mine = ring + warp * (G::STAGES * G::STAGE);
    float *pt = pts + (G::MMA16 ? 0 : warp * kBlock * 20);
    Feed<G> feed;
    feed.start(a, run, any, warp, lane);
    for (int s = 0; s < G::STAGES; ++s) feed.issue(a, &km, &vm, mine + s * G::STAGE, &full[warp][s], s, warp, lane);

    // ---- segments
    int it = 0;                        // tiles of this warp so far
    bool dead = false;
    for (bool more = any || a.cluster; more;) {
        const int hk = run.j / a.n_rb, rb = run.j - hk * a.n_rb;
        U u;
        if constexpr (G::Q != 0) {
            U::stage_queries(a, run.b, hk, rb, sq);
            __syncthreads();
        }
        u.begin(a, run.b, hk, rb, lane);
        for (int tile = run.begin + warp; tile < run.end; tile += G::WARPS, ++it) {
            const int s = it % G::STAGES;
            uint8_t *stage = mine + s * G::STAGE;
            if (!dead) {
                const bool came = ptx::mbar_wait(&full[warp][s], (it / G::STAGES) & 1, &gave_up);
                dead = __any_sync(0xffffffffu, !came);
                if (dead) {
                    gave_up = 1;
                    *a.status = GDN_ERR_TIMEOUT;
                }
            }
            if (dead) continue;
            u.tile(a, stage, sq, pt, tile * kTile, !(feed.bad >> s & 1u), lane);
            __syncwarp();
            feed.issue(a, &km, &vm, stage, &full[warp][s], s, warp, lane);
        }
        u.finish();

        // ---- the warps' parts of the segment join
        const int g = lane >> 2, t = lane & 3;
        const bool whole = run.begin == 0 && run.end == run.n;
        float *part_out = whole || a.cluster ? nullptr
                                             : a.ws + partial_slot(cta, run.begin == 0) * kPartial<G::ROWS, DV>;
        if (g == 0 && !(COLS && t >= 2))
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    sm[warp * G::ROWS + nb * kBlock + 2 * t + r] = u.m[nb][r];
                    sl[warp * G::ROWS + nb * kBlock + 2 * t + r] = u.l[nb][r];
                }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            if (!(COLS && t >= 2))
#pragma unroll
                for (int i = 0; i < U::MT; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        merge[(warp * kBlock + 2 * t + (e & 1)) * DV + U::element_of(i, e, g)] = u.o[nb][i][e];
            __syncthreads();
            constexpr int VALID = COLS ? 4 : kBlock;
            for (int x = tid; x < VALID * (DV / 4); x += G::THREADS) {
                const int r = x / (DV / 4), c = x - r * (DV / 4), row = nb * kBlock + r;
                float M = -INFINITY;
#pragma unroll
                for (int w = 0; w < G::WARPS; ++w) M = fmaxf(M, sm[w * G::ROWS + row]);
                float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
                float L = 0.f;
#pragma unroll
                for (int w = 0; w < G::WARPS; ++w) {
                    const float f = weight(sm[w * G::ROWS + row], M);
                    const float lw = sl[w * G::ROWS + row];
                    if (f != 0.f || lw != lw) {        // (a row of NaN scores has no maximum)
                        L = fmaf(f, lw, L);
                        y = fma4(f, *reinterpret_cast<const float4 *>(merge + (w * kBlock + r) * DV + 4 * c), y);
                    }
                }
                if (a.cluster > 1) {
                    *reinterpret_cast<float4 *>(merge + r * DV + 4 * c) = y;
                    if (c == 0) {
                        sm[G::WARPS * G::ROWS + row] = M;
                        sl[G::WARPS * G::ROWS + row] = L;
                    }
                } else if (part_out) {
                    *reinterpret_cast<float4 *>(part_out + row * DV + 4 * c) = y;
                    if (c == 0) {
                        part_out[G::ROWS * DV + row] = M;
                        part_out[G::ROWS * (DV + 1) + row] = L;
                    }
                } else {
                    write_out<DV>(a, run.b, hk, rb * G::ROWS + row, c, y, L);
                }
            }
            if (a.cluster > 1) {       // ... and the CTAs': each takes its share of the rows' elements
                cluster_sync();
                for (int x = rank * G::THREADS + tid; x < VALID * (DV / 4); x += a.cluster * G::THREADS) {
                    const int r = x / (DV / 4), c = x - r * (DV / 4), row = nb * kBlock + r;
                    float mk[kMaxCluster], M = -INFINITY, L = 0.f;
#pragma unroll
                    for (int p = 0; p < kMaxCluster; ++p) {
                        mk[p] = p < a.cluster ? peer_float(sm + G::WARPS * G::ROWS + row, p) : -INFINITY;
                        M = fmaxf(M, mk[p]);
                    }
                    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int p = 0; p < kMaxCluster; ++p) {
                        const float f = weight(mk[p], M);
                        if (p >= a.cluster) continue;
                        const float lp = peer_float(sl + G::WARPS * G::ROWS + row, p);
                        if (f != 0.f || lp != lp) {
                            L = fmaf(f, lp, L);
                            y = fma4(f, peer_float4(merge + r * DV + 4 * c, p), y);
                        }
                    }
                    write_out<DV>(a, run.b, hk, rb * G::ROWS + row, c, y, L);
                }
                cluster_sync();        // peers are done reading
            } else {
                __syncthreads();
            }
        }
        more = any && run.next(a);
    }
}

// Joins the parts of units that runs cut: block (c - 1, y) is for the unit that the boundary between runs c - 1
// and c cuts, if it is the first to cut it, and rows y, y + gridDim.y, ... of it.
constexpr int kJoinThreads = 256;
template <int ROWS, int DV>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const Attn a, const int warps) {
    constexpr int COLS4 = DV / 4, GROUPS = kJoinThreads / COLS4;           // groups of threads share a row's parts
    __shared__ int part[32], found[2];
    __shared__ float4 sums[kJoinThreads];
    __shared__ float sums_l[GROUPS];
    kv4::after_the_kernel_before();
    const int tid = threadIdx.x, lane = tid & 31;
    const int total = total_tiles(a, part, kJoinThreads);
    const int runs = runs_of(total, warps);
    const int c = (int)blockIdx.x + 1;
    if (c >= runs) return;
    const int cut = run_begin(total, runs, c);
    if (tid < 32) {
        int before;
        const int b = find_tile(a, cut, lane, &before);
        if (lane == 0) {
            found[0] = b;
            found[1] = before;
        }
    }
    __syncthreads();
    const int b = found[0], n = tiles_at(a, b);
    const int j = (cut - found[1]) / n, first = found[1] + j * n;
    if (cut == first) return;
    const int r0 = run_of(total, runs, first), r1 = run_of(total, runs, first + n - 1);
    if (c != r0 + 1) return;
    const int hk = j / a.n_rb, rb = j - hk * a.n_rb, parts = r1 - r0 + 1;
    const int group = tid / COLS4, col = tid - group * COLS4;
    // part p: of run r0 + p; the unit begins in run r0
    auto at = [&](int p) { return a.ws + partial_slot(r0 + p, p == 0) * kPartial<ROWS, DV>; };
    for (int row = (int)blockIdx.y; row < ROWS && rb * ROWS + row < a.R; row += gridDim.y) {
        float M = -INFINITY;
        for (int p = lane; p < parts; p += 32) M = fmaxf(M, at(p)[ROWS * DV + row]);
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        float L = 0.f;
#pragma unroll 4
        for (int p = group; p < parts; p += GROUPS) {
            const float *q = at(p);
            const float m = q[ROWS * DV + row], l = q[ROWS * (DV + 1) + row];
            const float4 x = *reinterpret_cast<const float4 *>(q + row * DV + 4 * col);
            const float f = weight(m, M);
            if (f != 0.f || l != l) {
                L = fmaf(f, l, L);
                y = fma4(f, x, y);
            }
        }
        sums[tid] = y;
        if (col == 0) sums_l[group] = L;
        __syncthreads();
        if (group == 0) {
            for (int k = 1; k < GROUPS; ++k) {
                y = fma4(1.f, sums[k * COLS4 + col], y);
                L += sums_l[k];
            }
            write_out<DV>(a, b, hk, rb * ROWS + row, col, y, L);
        }
        __syncthreads();
    }
}

template <typename T, int DK, int DV, int NB, bool COLS>
cudaError_t launch_one(const CUtensorMap &km, const CUtensorMap &vm, const Attn &a, int grid, cudaStream_t stream) {
    using G = Geo<T, DK, DV, NB>;
    static PerDeviceOnce setup;
    cudaError_t e = setup.run([] {
        return cudaFuncSetAttribute(attn_kernel<T, DK, DV, NB, COLS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    G::SMEM);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.cluster ? a.cluster : 1;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(G::THREADS);
    cfg.dynamicSmemBytes = G::SMEM;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, attn_kernel<T, DK, DV, NB, COLS>, km, vm, a);
    if (e != cudaSuccess || a.cluster || grid < 2) return e;
    const int rows = a.R < G::ROWS ? a.R : G::ROWS;
    return kv4::launch_early(join_kernel<G::ROWS, DV>, dim3((unsigned)grid - 1, (unsigned)(rows < 8 ? rows : 8)),
                             kJoinThreads, 0, stream, a, G::WARPS);
}

template <typename T, int DK, int DV>
cudaError_t launch_rows(const CUtensorMap &km, const CUtensorMap &vm, const Attn &a, int grid, cudaStream_t stream) {
    if constexpr (sizeof(T) == 4) {
        return launch_one<T, DK, DV, 1, false>(km, vm, a, grid, stream);
    } else {
        constexpr bool wide = DK > 128 || DV > 128;
        // of at most 4 rows, the weights' remainders enter in the free columns of the same MMAs
        if (a.R <= 4) return launch_one<T, DK, DV, 1, true>(km, vm, a, grid, stream);
        switch (blocks_of(wide, false, a.R)) {
            case 1: return launch_one<T, DK, DV, 1, false>(km, vm, a, grid, stream);
            case 2: return launch_one<T, DK, DV, 2, false>(km, vm, a, grid, stream);
            default:
                if constexpr (!wide) return launch_one<T, DK, DV, 4, false>(km, vm, a, grid, stream);
                return cudaErrorInvalidValue;
        }
    }
}

}  // namespace

template <typename T, int DK>
cudaError_t launch_attn(int dv, const CUtensorMap &km, const CUtensorMap &vm, const Attn &a, int grid,
                        cudaStream_t stream) {
    switch (dv) {
        case 64: return launch_rows<T, DK, 64>(km, vm, a, grid, stream);
        case 128: return launch_rows<T, DK, 128>(km, vm, a, grid, stream);
        case 256: return launch_rows<T, DK, 256>(km, vm, a, grid, stream);
        default: return cudaErrorInvalidValue;
    }
}
template cudaError_t launch_attn<GDN_PAGED_ATTN_T, GDN_PAGED_ATTN_DK>(int, const CUtensorMap &, const CUtensorMap &,
                                                                      const Attn &, int, cudaStream_t);
#endif  // GDN_PAGED_ATTN_T

}  // namespace paged
}  // namespace gdn
