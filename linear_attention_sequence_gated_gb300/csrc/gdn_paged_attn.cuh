// Decode attention over a paged cache of 16- or 32-bit rows (gdn_flash_attn_paged): for
// every sequence b, query head h and query i,
//     out[b, i, h, :] = softmax_j(scale q[b,h,i] . k[b,hk,j] + mask[b,0,i,j]) v[b,hk,j,:]
// over the tokens j that the sequence holds (with `causal`, up to the query's own), hk = h /
// (n_heads / n_heads_kv), row j of sequence b in page table[b][j / page] at j % page.
//
// The cache is streamed once: (dk + dv) e bytes a token and kv head against 2 (dk + dv) flops
// a row = (query head of the group, query), so HBM bounds calls of few rows and the kernel's work is to keep copies in
// flight; from about 24 rows the warps' instructions do.
//   * A tile is 16 tokens of one kv head, which never leave a page.  Four warps stream a CTA's tiles through
//     a ring in shared memory, by TMA boxes of 16 tokens x 128 bytes with 128-byte swizzling (any order of a
//     cache's tokens and heads: the tensor map holds the strides), whose rows ldmatrix reads without bank
//     conflicts.  (One such warp takes 700 cycles a tile: the table's entry, its address, four to eight boxes.)
//   * Each tile goes to one group of the 8 or 12 warps that compute, where every warp takes another 8 rows.  Those
//     warps get the registers that the others give up.
//   * 16-bit rows: S^T = K Q^T (M = 16 tokens, N = 8 rows) and O^T += V^T P^T (M = 16 elements,
//     N = 8 rows, K = 16 tokens) by m16n8k16 MMAs with fp32 accumulators, the weights as two terms of f16 (22 bits) or
//     three of bf16 (24), transposed in registers by movmatrix.  Up to 4
//     rows, the second terms stand in the columns that no row needs.
//   * fp32 rows: the same by m16n8k8 tf32 MMAs, each operand as hi + lo (11 bits each), three products.
//   * Scores, maxima, sums and outputs are fp32; each tile's products reach the outputs by one
//     fp32 FMA, since the MMAs' own accumulation truncates.
//
// Work is shared out in tiles, not in sequences: the tiles of all units (sequence, kv head, block
// of rows) in a row are cut into equal runs, one a CTA, so ragged batches and single long
// sequences load the GPU evenly.  The groups of a CTA take the tiles of a unit in turn and join
// their parts in shared memory at its end, while the next unit's copies are in flight.  A unit
// that runs cut leaves (max, sum, output) in the workspace, and a second kernel joins those parts
// in a fixed order.  A call of few tiles gives each unit a cluster of CTAs instead, which join
// through distributed shared memory: one launch, no workspace.
//
// Measured (GPU time of captured calls): 64 sequences x 32/8 heads x 4096 tokens x 128, bf16: 165 - 169 us, 94 - 96 % of the
// rate of a copy; 2 x 16/4 x (100003, 50001) x 128: 55 us, 82 % (runs start, fill, drain and join in about 9 us); 16 x 5 queries x 32/8 x
// up to 5001 x 128, f16: 45 us, of which the stream alone takes 39; 64 queries' rows a kv head there: 102 us, the stream alone
// (two units, each tile twice) 62, at 30 % of the tensor pipe and half of all issue slots.
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
constexpr int kUnitCost = 16;           // tiles that beginning and ending a unit counts for when runs are cut

struct Attn {
    const void *q, *mask;
    void *out;
    float *ws;
    const int *table, *lens;
    int *status;
    long long q_seq, q_head, q_query;  // in elements
    int n_seqs, H, Hkv, n_q, R, n_rb;  // R rows a kv head in n_rb units,
    int blocks, groups;                // each of `blocks` blocks of 8, one a warp of each of a CTA's groups
    int ring;                          // stages of the ring
    int n_pages, tpp, max_pages;       // tpp: tiles of a page
    float scale;
    int out_type;
    int cluster, cluster_log;          // CTAs a unit (a power of two), or 0: equal runs
    int rep;                           // H / Hkv
    Divisor by_q, by_rb, by_tpp, by_units;     // n_q, n_rb, tpp, units of a sequence
    bool causal;
    int k_order, v_order;              // of the tensor maps' outer coordinates: two bits each, 0 token, 1 head, 2 page
};

// Shared memory of the kernel for widths dk and dv, rows of elt bytes and `warps` warps, each with a block of 8 rows at
// a time, `most` different ones at most.
struct Room {
    int columns;                       // the warps' outputs are joined so many columns at a time,
    int merge;                         // in rows padded against bank conflicts
    int weights, sums;                 // fp32 weights on their way to B operands; maxima and sums
    int q_row, q_block;                // fp32 queries as hi and lo, in padded rows; bytes of a block (16-bit ones are
                                       // in registers)
    int pool;                          // bytes for the ring and the queries
};
constexpr int kSmemMax = 227 * 1024;
constexpr Room room_of(int dk, int dv, int elt, int warps, int most) {
    const int limit = (elt == 2 ? 32 : 16) * 1024, row = warps * kBlock * 4;
    Room r{};
    r.columns = row * (dv + 4) <= limit ? dv : dv > 128 && row * 132 <= limit ? 128 : 64;
    r.merge = row * (r.columns + 4);
    r.weights = elt == 2 ? 0 : warps * kBlock * 20 * 4;
    r.sums = 2 * (warps + most) * kBlock * 4;
    r.q_row = dk * 8 + 64;
    r.q_block = elt == 2 ? 0 : kBlock * r.q_row;
    // (1 KB for the ring's alignment, 3 KB for barriers and the like)
    r.pool = (kSmemMax - 4096 - r.merge - r.weights - r.sums) / 16 * 16;
    return r;
}
constexpr int kMaxRing = 48;

// How the rows of a kv head and the warps of a CTA are shared out.  Tiles go round the groups of warps; each
// warp of a group takes another block of 8 rows of the same tile, so that the cache is read once for all of them:
// 12 warps where 152 registers hold a block's output, else 8, as so many groups as there are blocks and tiles for.
// Four more warps fill the ring.
// A stage of the ring is filled by one warp and, within a segment, emptied by one group only, so the
// ring is a whole number of tiles a group: a barrier's parity tells a phase from the next, but not from the
// one after, so whoever waits for a stage has to have seen its last use end.
struct Share {
    int warps, most;                   // warps that compute; blocks of rows of a unit at most
    int blocks, groups, units;         // blocks of a unit, groups of so many warps, units of a kv head
    int ring;                          // stages
};
constexpr int kFillers = 4;
constexpr Share share_of(int dk, int dv, int elt, int R) {
    const bool wide = elt == 4 || dk > 128 || dv > 128;
    const int warps = wide ? 8 : 12, most = !wide ? 6 : elt == 2 || R > kBlock ? 4 : 1;
    const int all = (R + kBlock - 1) / kBlock, units = (all + most - 1) / most, blocks = (all + units - 1) / units;
    const Room room = room_of(dk, dv, elt, warps, most);
    int tiles = (room.pool - blocks * room.q_block) / (kTile * (dk + dv) * elt);
    if (tiles > kMaxRing) tiles = kMaxRing;
    const int groups = warps / blocks < tiles ? warps / blocks : tiles;
    return {warps, most, blocks, groups, units, tiles - tiles % groups};
}

// A run that covers a unit in part leaves a partial result in the workspace: [rows][dv] outputs, [rows] maxima,
// [rows] sums, so many floats.
__host__ __device__ inline size_t partial_size(int rows, int dv) { return (size_t)rows * (dv + 2); }

// The kernel for rows of type T and keys of width DK (one translation unit each).
template <typename T, int DK>
cudaError_t launch_attn(int dv, const CUtensorMap &km, const CUtensorMap &vm, const Attn &a, int grid,
                        cudaStream_t stream);

#ifdef GDN_PAGED_ATTN_T
namespace {

using kv4::run_begin;
using kv4::run_of;
using kv4::partial_slot;

// Shape of the kernel for widths DK and DV, type T, WARPS warps and up to MOST blocks of rows.
template <typename T, int DK, int DV, int WARPS, int MOST>
struct Geo {
    static constexpr int E = (int)sizeof(T);
    static constexpr bool MMA16 = E == 2;
    static constexpr int BOX = 128 / E;                // elements of a box's row
    static constexpr int KB = kTile * DK * E, VB = kTile * DV * E, STAGE = KB + VB;
    static constexpr int THREADS = WARPS * 32, ALL = THREADS + 32 * kFillers;
    // Registers a thread: the launch's, and after the warps that fill the ring have given theirs up.  (Those keep 72 beside
    // 16-bit rows of 256, which spill with 56: 8 x 16/2 heads x 4000 x 256 f16 28.7 and 31.6 us; fp32 rows need the 224.)
    static constexpr int REGS = WARPS == 12 ? 128 : 168;
    static constexpr int FILL_REGS = WARPS == 12 || E == 4 ? 56 : 72, WORK_REGS = WARPS == 12 ? 152 : E == 4 ? 224 : 216;
    static_assert(WARPS % 4 == 0 && THREADS * WORK_REGS + 32 * kFillers * FILL_REGS <= ALL * REGS,
                  "a split of more registers than the launch has would wait forever");
    static constexpr Room R = room_of(DK, DV, E, WARPS, MOST);
    static constexpr int MC = R.columns, QROW = R.q_row;
    static constexpr int QBLOCK = R.q_block, RING = R.pool - MOST * QBLOCK;    // (the least that a ring has)
    static constexpr int SMEM = 1024 + R.pool + R.merge + R.weights + R.sums;
    static_assert(RING / STAGE >= 4, "ring");
    static_assert(17 * kMaxRing + 160 + (8 + 4 * kMaxCluster) * MOST * kBlock <= (3 << 10), "barriers and the like");
    static_assert(R.merge % 16 == 0 && QROW % 16 == 0 && R.weights % 16 == 0 && DV % MC == 0, "alignment");
    static_assert(WARPS * kBlock * (DV + 4) * 4 <= RING / STAGE / 4 * 4 * STAGE, "the last unit is joined in the ring");
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
// the same with zero accumulators
template <typename T>
__device__ __forceinline__ void mma0(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
            "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
    else if constexpr (std::is_same<T, __half>::value)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
            "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
    else
        asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 "
            "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// 8 x 8 transpose of 16-bit elements across the warp: lane (g, t) gives row g, columns 2t,
// 2t + 1 and gets row g of the transpose.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// (x, y) as a 16-bit pair, and what is left of them
template <typename T>
__device__ __forceinline__ uint32_t round2(float &x, float &y) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        const float2 f = __bfloat1622float2(h);
        x -= f.x;
        y -= f.y;
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __half2 h = __floats2half2_rn(x, y);
        const float2 f = __half22float2(h);
        x -= f.x;
        y -= f.y;
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}
// fp32 as tf32 hi + lo, 11 bits each.  hi is cut off behind 0.36 to 0.72 of its last bit, added by a product that rounds
// toward zero: it stays finite up to the largest numbers, and lo, of either sign, is 0.72 of that bit at most, so few
// lose more than one bit to its own cut: x is off by 3 * 2^-23 at most, 2^-24 in the root mean square.  (hi to nearest: 2^-23
// and 0.7 * 2^-24, but 2^128 for the largest unless held back.  16 x 16 queries x 32/8 x 5001 x 128, us: so 527; to nearest
// unprotected 518, by a minimum 596, by adding half of the last bit toward zero 580, by the conversion 692.)
// A NaN's lo is NaN; so is an infinity's.
__device__ __forceinline__ void split_tf32(float x, uint32_t &hi, uint32_t &lo) {
    hi = __float_as_uint(__fmul_rz(x, 1.f + 0.36f * 0x1p-10f)) & 0xffffe000u;
    lo = __float_as_uint(x - __uint_as_float(hi)) & 0xffffe000u;
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

// Behind the partial results of all runs: which unit a run leaves to those after it, and in how many parts it lies.
struct Open {
    int b, j, parts, unused;
};
__device__ __forceinline__ Open *open_of(const Attn &a, int grid, int dv) {
    return reinterpret_cast<Open *>(a.ws + 2 * grid * partial_size(a.blocks * kBlock, dv));
}

// Sum of x over the block, in every thread; `part` is 32 ints, free again after the next barrier.
__device__ __forceinline__ int block_sum(int x, int *part, int warps) {
    x = __reduce_add_sync(0xffffffffu, x);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    return __reduce_add_sync(0xffffffffu, lane < warps ? part[lane] : 0);
}

// Sum of x over this lane and those before it.
__device__ __forceinline__ int warp_sum(int x, int lane) {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += o;
    }
    return x;
}

// Steps of a unit of n tiles: the first kUnitCost stand for its beginning and end.
__device__ __forceinline__ int steps_of(int n) { return n ? n + kUnitCost : 0; }

// Steps of all units; a length beyond the table shows in the status word.
__device__ __forceinline__ int total_steps(const Attn &a, int *part, int threads) {
    int n = 0;
    for (int b = threadIdx.x; b < a.n_seqs; b += threads) {
        n += steps_of(tiles_at(a, b));
        if (a.lens[b] > capacity(a)) *a.status = GDN_ERR_PAGE;
    }
    return block_sum(n, part, threads / 32) * units_of(a);
}

// Whole warp: the sequence that step x of all lies in, and the steps before it.
__device__ __forceinline__ int find_step(const Attn &a, int x, int lane, int *before) {
    int done = 0;
    for (int base = 0;; base += 32) {
        const int n = base + lane < a.n_seqs ? steps_of(tiles_at(a, base + lane)) * units_of(a) : 0;
        const int incl = done + warp_sum(n, lane);
        const unsigned hit = __ballot_sync(0xffffffffu, incl > x);
        if (hit || base + 32 >= a.n_seqs) {            // (x is below the total, so there is one)
            const int src = hit ? __ffs(hit) - 1 : 31;
            *before = __shfl_sync(0xffffffffu, incl - n, src);
            return min(base + src, a.n_seqs - 1);
        }
        done = __shfl_sync(0xffffffffu, incl, 31);
    }
}

// Runs of a call of T steps: fewer where they would have less than a tile for each group.
__device__ __forceinline__ int runs_of(const Attn &a, int T) { return min(kGrid, (T + a.groups - 1) / a.groups); }

// A walk over the units of a CTA's run: a segment is the part of a unit that lies in it.
struct Walk {
    int left;                          // steps of the run from this segment on
    int b, j;                          // sequence, unit in it
    int from, to;                      // steps of the unit, and
    int begin, end, n;                 // tiles [begin, end) of its n
    int raw;                           // the sequence's length
    __device__ __forceinline__ void set(const Attn &a) {
        raw = max(a.lens[b], 0);
        n = (min(raw, capacity(a)) + kTile - 1) / kTile;
    }
    __device__ __forceinline__ bool cut() {
        to = min(n + kUnitCost, from + left);
        begin = max(from - kUnitCost, 0);
        end = max(to - kUnitCost, 0);
        return begin < end;
    }
    __device__ __forceinline__ bool next(const Attn &a) {
        left -= to - from;
        if (left <= 0) return false;
        from = 0;
        if (++j == units_of(a)) {
            j = 0;
            do {
                if (++b >= a.n_seqs) return false;
                set(a);
            } while (n == 0);
        }
        return cut();                  // (a run may end within a unit's first steps)
    }
};

// One warp's share of one unit: an online softmax of 8 rows over tiles.
template <typename T, int DK, int DV, typename G, bool COLS>
struct Unit {
    static constexpr bool MMA16 = G::MMA16;
    static constexpr int KS = DK / 16, MT = DV / 16;   // 16-element steps of a key, blocks of a value row
    // weights of f16 rows are scaled by 2^12, so that small ones keep their bits
    static constexpr float kBits = std::is_same<T, __half>::value ? 12.f : 0.f;

    uint32_t qf[MMA16 ? KS : 1][2];
    float m[2], l[2];                  // of rows 2t, 2t + 1: running maximum, this lane's sum of weights
    float o[MT][4];
    int qi[2];                         // the row's query; -1: no such row
    int raw, all, len;                 // length; tokens that every row sees and no mask changes; in the table
    int b;

    __device__ __forceinline__ static const T *q_row(const Attn &a, int b, int hk, int row) {
        const int h = a.by_q.into(row), i = row - h * a.n_q;
        return static_cast<const T *>(a.q) + b * a.q_seq + (hk * a.rep + h) * a.q_head + i * a.q_query;
    }

    // fp32 queries of the unit's blocks to shared memory, by the whole CTA (a barrier follows).
    __device__ __forceinline__ static void stage_queries(const Attn &a, int b, int hk, int row0, uint8_t *sq) {
        for (int x = threadIdx.x; x < a.blocks * kBlock * (DK / 4); x += G::THREADS) {
            const int r = x / (DK / 4), c = x - r * (DK / 4);
            uint4 w = make_uint4(0, 0, 0, 0), hi, lo;
            if (row0 + r < a.R) w = *reinterpret_cast<const uint4 *>(q_row(a, b, hk, row0 + r) + c * 4);
            split_tf32(__uint_as_float(w.x), hi.x, lo.x);
            split_tf32(__uint_as_float(w.y), hi.y, lo.y);
            split_tf32(__uint_as_float(w.z), hi.z, lo.z);
            split_tf32(__uint_as_float(w.w), hi.w, lo.w);
            *reinterpret_cast<uint4 *>(sq + r * G::QROW + c * 16) = hi;
            *reinterpret_cast<uint4 *>(sq + r * G::QROW + DK * 4 + c * 16) = lo;
        }
    }

    // 16-bit queries of rows row0 .. row0 + 7 of kv head hk, as B operands.
    __device__ __forceinline__ static void load_queries(const Attn &a, const Walk &w, int row0, int lane,
                                                        uint32_t (&q)[MMA16 ? KS : 1][2]) {
        if constexpr (MMA16) {
            // (a row that is not there takes the last one's, for columns that nobody reads: nothing here may wait
            // for the loads)
            const int g = lane >> 2, t = lane & 3, row = min(COLS ? g & 3 : row0 + g, a.R - 1);
            const uint32_t *p = reinterpret_cast<const uint32_t *>(q_row(a, w.b, a.by_rb.into(w.j), row)) + t;
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                q[s][0] = p[s * 8];
                q[s][1] = p[s * 8 + 4];
            }
        }
    }
    __device__ __forceinline__ void begin(const Attn &a, const Walk &w, int row0, int lane) {
        const int t = lane & 3;
        b = w.b;
        raw = w.raw;
        len = min(raw, capacity(a));
        all = a.mask ? 0 : a.causal ? min(len, max(raw - a.n_q + 1, 0)) : len;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = COLS ? (2 * t + r) & 3 : row0 + 2 * t + r;
            qi[r] = row < a.R ? row - a.by_q.into(row) * a.n_q : -1;
            m[r] = -INFINITY;
            l[r] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    }

    // S^T of a tile: entry e is token g + 8 (e >> 1) and row 2t + (e & 1).
    __device__ __forceinline__ void scores(uint32_t k, const uint8_t *sq, int lane, float (&s)[4]) const {
        const int g = lane >> 2, t = lane & 3;
        if constexpr (MMA16) {
            const uint32_t row = k + (lane & 15) * 128, x = lane & 7, half = lane >> 4;
            float d[4][4];             // four chains of products: one alone waits for each product's latency
#pragma unroll
            for (int c = 0; c < KS; ++c) {
                uint32_t A[4];
                ldsm4(A, row + (c >> 2) * 2048 + (((2 * (c & 3) + half) ^ x) << 4));
                if (c < 4) mma0<T>(d[c], A, qf[c][0], qf[c][1]);
                else mma<T>(d[c & 3], A, qf[c][0], qf[c][1]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) s[e] = (d[0][e] + d[1][e]) + (d[2][e] + d[3][e]);
        } else {
            // Lane (g, t) has elements 4t .. 4t + 3 of each 16 of tokens g and g + 8: the first two
            // are columns t and t + 4 of one k8 product, the others of the next (the queries' likewise).
            // Odd g read the second 16 of each 32 first, so that 8 lanes read 8 different pieces.
            const uint32_t ra = k + g * 128, x = g & 7, odd = g & 1;
            const uint8_t *q = sq + g * G::QROW + t * 16;
            float d[6][4];             // chains of products: hi hi, lo hi, hi lo of the first and second 16
#pragma unroll
            for (int n = 0; n < 6; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) d[n][e] = 0.f;
#pragma unroll 2
            for (int c = 0; c < DK / 32; ++c) {
                const uint32_t p0 = ra + c * 2048 + (((t + 4 * odd) ^ x) << 4);
                const uint32_t p1 = ra + c * 2048 + (((t + 4 * (odd ^ 1)) ^ x) << 4);
                const uint4 u0 = lds16(p0), u1 = lds16(p1), v0 = lds16(p0 + 1024), v1 = lds16(p1 + 1024);
                uint4 qh[2], ql[2];
                uint32_t hi[2][2][4], lo[2][2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint4 u = h == (int)odd ? u0 : u1, v = h == (int)odd ? v0 : v1;
                    qh[h] = *reinterpret_cast<const uint4 *>(q + c * 128 + h * 64);
                    ql[h] = *reinterpret_cast<const uint4 *>(q + DK * 4 + c * 128 + h * 64);
                    split_tf32(__uint_as_float(u.x), hi[h][0][0], lo[h][0][0]);
                    split_tf32(__uint_as_float(v.x), hi[h][0][1], lo[h][0][1]);
                    split_tf32(__uint_as_float(u.y), hi[h][0][2], lo[h][0][2]);
                    split_tf32(__uint_as_float(v.y), hi[h][0][3], lo[h][0][3]);
                    split_tf32(__uint_as_float(u.z), hi[h][1][0], lo[h][1][0]);
                    split_tf32(__uint_as_float(v.z), hi[h][1][1], lo[h][1][1]);
                    split_tf32(__uint_as_float(u.w), hi[h][1][2], lo[h][1][2]);
                    split_tf32(__uint_as_float(v.w), hi[h][1][3], lo[h][1][3]);
                }
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t h0 = n ? qh[h].z : qh[h].x, h1 = n ? qh[h].w : qh[h].y;
                        const uint32_t l0 = n ? ql[h].z : ql[h].x, l1 = n ? ql[h].w : ql[h].y;
                        mma<T>(d[3 * h], hi[h][n], h0, h1);
                        mma<T>(d[3 * h + 1], lo[h][n], h0, h1);
                        mma<T>(d[3 * h + 2], hi[h][n], l0, l1);
                    }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) s[e] = ((d[1][e] + d[4][e]) + (d[2][e] + d[5][e])) + (d[0][e] + d[3][e]);
        }
    }

    // Element of a value row that o[i][e] sums, and where the stage holds it.
    __device__ __forceinline__ static int element_of(int i, int e, int g) {
        return MMA16 ? i * 16 + g + 8 * (e >> 1) : (i >> 1) * 32 + 4 * g + 2 * (i & 1) + (e >> 1);
    }
    __device__ __forceinline__ static uint32_t value_at(int tok, int x) {
        return (uint32_t)((x / G::BOX) * 2048 + tok * 128 + ((((x % G::BOX) * G::E / 16) ^ (tok & 7)) << 4) +
                          x * G::E % 16);
    }

    // Values of tokens that some row must not see may be anything, infinities and NaN among them, and
    // a weight of 0 does not silence those in a product.  Where such a tile has any, its values are taken
    // one by one by the rows that see them.  (p: weights, x: scores.)
    __device__ __forceinline__ void odd_values(const uint8_t *v, const float (&p)[4], const float (&x)[4], int lane) {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll 1
        for (int tok = 0; tok < kTile; ++tok) {
            const int src = (tok & 7) * 4 + t;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float w0 = __shfl_sync(0xffffffffu, p[r], src), w1 = __shfl_sync(0xffffffffu, p[r + 2], src);
                const float x0 = __shfl_sync(0xffffffffu, x[r], src), x1 = __shfl_sync(0xffffffffu, x[r + 2], src);
                const float w = tok < 8 ? w0 : w1, sc = tok < 8 ? x0 : x1;
                if (sc == -INFINITY || (COLS && t >= 2)) continue;
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int e = r; e < 4; e += 2) {
                        const float y = to_float<T>(*reinterpret_cast<const T *>(v + value_at(tok, element_of(i, e, g))));
                        o[i][e] = fmaf(w, y, o[i][e]);
                    }
            }
        }
    }
    // Whether any value of the tile is not finite: 0 times it is NaN.
    __device__ __forceinline__ static bool any_odd(const uint8_t *v, int lane) {
        if constexpr (MMA16) {
            const uint32_t at = ptx::smem_u32(v) + ((lane & 7) + ((lane >> 4) << 3)) * 128, sw = lane & 7, half = (lane >> 3) & 1;
            float d[2][4] = {};
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                uint32_t A[4];
                ldsm4_t(A, at + (i >> 2) * 2048 + (((2 * (i & 3) + half) ^ sw) << 4));
                mma<T>(d[i & 1], A, 0u, 0u);
            }
            float sum = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) sum += d[0][e] + d[1][e];
            return __any_sync(0xffffffffu, sum != sum);
        } else {
            float acc[4] = {};
#pragma unroll 4
            for (int i = 0; i < G::VB / 512; ++i) {
                const uint4 w = *reinterpret_cast<const uint4 *>(v + (i * 32 + lane) * 16);
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[e] = fmaf(__uint_as_float(u[e]), 0.f, acc[e]);
            }
            const float sum = (acc[0] + acc[1]) + (acc[2] + acc[3]);
            return __any_sync(0xffffffffu, sum != sum);
        }
    }

    // The tile in `stage`, tokens pos .. pos + 15 of the sequence.
    __device__ __forceinline__ void tile(const Attn &a, const uint8_t *stage, int pos, const uint8_t *sq, float *pt, int lane) {
        const int g = lane >> 2, t = lane & 3;
        float s[4], x[4], cf[2], add[4];
        // tokens of the tile, from this lane's on, that a row sees
        auto seen = [&](int r) {
            return (qi[r] < 0 ? 0 : a.causal ? min(len, raw - a.n_q + 1 + qi[r]) : len) - pos - g;
        };
        if (a.mask)                    // loaded ahead of the products
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const T *p = static_cast<const T *>(a.mask) + ((size_t)b * a.n_q + qi[r]) * (size_t)capacity(a) + pos + g;
                add[r] = seen(r) > 0 ? to_float<T>(p[0]) : -INFINITY;
                add[r + 2] = seen(r) > 8 ? to_float<T>(p[8]) : -INFINITY;
            }
        scores(ptx::smem_u32(stage), sq, lane, s);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = s[e] * a.scale;
        const bool plain = pos + kTile <= all;
        if (!plain) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (a.mask) x[e] = add[e] == -INFINITY ? -INFINITY : x[e] + add[e];
                else if (seen(e & 1) <= 8 * (e >> 1)) x[e] = -INFINITY;
            }
        }
        float mx[2] = {fmaxf(x[0], x[2]), fmaxf(x[1], x[3])};
#pragma unroll
        for (int off = 4; off < 32; off <<= 1)
#pragma unroll
            for (int r = 0; r < 2; ++r) mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], off));
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            // Weights go by differences, 2^((x - maximum) log2 e), which are exact where they matter:
            // masks of the type's lowest value and scores of any size keep their order, and the factor of
            // earlier tiles is exactly 1 while the maximum stands.
            const float old = m[r], mn = fmaxf(old, mx[r]), base = mn == -INFINITY ? 0.f : mn;
            m[r] = mn;
            cf[r] = exp2_approx((old - base) * kLog2e);
            s[r] = exp2_approx(fmaf(x[r] - base, kLog2e, kBits));
            s[r + 2] = exp2_approx(fmaf(x[r + 2] - base, kLog2e, kBits));
            l[r] = fmaf(l[r], cf[r], s[r] + s[r + 2]);
        }
        if (!plain && any_odd(stage + G::KB, lane)) {
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][e] *= cf[e & 1];
            odd_values(stage + G::KB, s, x, lane);
            return;
        }
        if constexpr (MMA16) {
            // Weights as 16-bit terms, largest first: two of f16 (22 bits), three of bf16 (24; two, 16 bits, would show in
            // outputs of bf16: one value in a thousand rounded to its neighbour).  In COLS the second stands in columns
            // 4 .. 7 of the first's products, where the rows' queries stand again.
            constexpr bool third = std::is_same<T, __nv_bfloat16>::value;
            uint32_t p1[2], p2[2], p3[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float y = s[2 * h], z = s[2 * h + 1];
                p1[h] = round2<T>(y, z);
                p2[h] = round2<T>(y, z);
                if constexpr (third) p3[h] = round2<T>(y, z);
                if constexpr (COLS) {
                    p1[h] = t >= 2 ? p2[h] : p1[h];
                    if constexpr (third) p2[h] = t >= 2 ? 0u : p3[h];
                }
                p1[h] = transpose8(p1[h]);
                if (!COLS || third) p2[h] = transpose8(p2[h]);
                if (!COLS && third) p3[h] = transpose8(p3[h]);
            }
            const uint32_t tok = (lane & 7) + ((lane >> 4) << 3);
            const uint32_t row = tok * 128 + G::KB, sw = lane & 7, half = (lane >> 3) & 1;
            // four blocks of 16 elements at a time, whose products do not wait for one another
#pragma unroll
            for (int i0 = 0; i0 < MT; i0 += 4) {
                float d[4][4];
                uint32_t A[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    ldsm4_t(A[i], ptx::smem_u32(stage) + row + (i0 >> 2) * 2048 + (((2 * i + half) ^ sw) << 4));
                // small terms first
                if (!COLS && third)
#pragma unroll
                    for (int i = 0; i < 4; ++i) mma0<T>(d[i], A[i], p3[0], p3[1]);
                if (!COLS || third)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (COLS || !third) mma0<T>(d[i], A[i], p2[0], p2[1]);
                        else mma<T>(d[i], A[i], p2[0], p2[1]);
                    }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (COLS && !third) mma0<T>(d[i], A[i], p1[0], p1[1]);
                    else mma<T>(d[i], A[i], p1[0], p1[1]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[i0 + i][e] = fmaf(o[i0 + i][e], cf[e & 1], d[i][e]);
            }
        } else {
            const uint32_t v = ptx::smem_u32(stage) + G::KB;
            // weights to [row][token]; lane (g, t) takes row g, tokens 2t, 2t + 1, 2t + 8, 2t + 9
            pt[(2 * t) * 20 + g] = s[0];
            pt[(2 * t + 1) * 20 + g] = s[1];
            pt[(2 * t) * 20 + g + 8] = s[2];
            pt[(2 * t + 1) * 20 + g + 8] = s[3];
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
                float d[2][2][4];      // of two M tiles: products of lo parts, and of hi ones
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t hi[2][4], lo[2][4];
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        split_tf32(__uint_as_float(w[2 * n][2 * i]), hi[n][0], lo[n][0]);
                        split_tf32(__uint_as_float(w[2 * n][2 * i + 1]), hi[n][1], lo[n][1]);
                        split_tf32(__uint_as_float(w[2 * n + 1][2 * i]), hi[n][2], lo[n][2]);
                        split_tf32(__uint_as_float(w[2 * n + 1][2 * i + 1]), hi[n][3], lo[n][3]);
                    }
                    mma0<T>(d[i][0], lo[0], ph[0], ph[1]);
                    mma0<T>(d[i][1], hi[0], ph[0], ph[1]);
                    mma<T>(d[i][0], lo[1], ph[2], ph[3]);
                    mma<T>(d[i][1], hi[1], ph[2], ph[3]);
                    mma<T>(d[i][0], hi[0], pl[0], pl[1]);
                    mma<T>(d[i][0], hi[1], pl[2], pl[3]);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[2 * c + i][e] = fmaf(o[2 * c + i][e], cf[e & 1], d[i][0][e] + d[i][1][e]);
            }
            __syncwarp();
        }
    }

    // Sums over the lanes that share rows; in COLS, the other columns' terms.
    __device__ __forceinline__ void finish() {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1)
#pragma unroll
            for (int r = 0; r < 2; ++r) l[r] += __shfl_xor_sync(0xffffffffu, l[r], off);
        if constexpr (COLS) {
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][e] += __shfl_xor_sync(0xffffffffu, o[i][e], 2);
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

// Over the 16 lanes of half a warp
__device__ __forceinline__ float max16(float x) {
#pragma unroll
    for (int off = 1; off < 16; off <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
    return x;
}
__device__ __forceinline__ float sum16(float x) {
#pragma unroll
    for (int off = 1; off < 16; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

// Which row of the output, (n_seqs, n_q, n_heads), belongs to row `row` of (b, hk)
__device__ __forceinline__ long long out_row(const Attn &a, int b, int hk, int row) {
    const int h = a.by_q.into(row), i = row - h * a.n_q;
    return ((long long)b * a.n_q + i) * a.H + hk * a.rep + h;
}

template <typename T, int DK, int DV, int WARPS, int MOST, bool COLS>
__global__ void __launch_bounds__(WARPS * 32 + 32 * kFillers, 1)
attn_kernel(const __grid_constant__ CUtensorMap km, const __grid_constant__ CUtensorMap vm, const Attn a) {
    using G = Geo<T, DK, DV, WARPS, MOST>;
    using Part = Unit<T, DK, DV, G, COLS>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = smem_raw + (-ptx::smem_u32(smem_raw) & 1023u);
    uint8_t *sq = ring + a.ring * G::STAGE;            // queries, behind the ring
    float *merge = reinterpret_cast<float *>(ring + G::R.pool);            // [WARPS][8][MC + 4]
    float *pts = reinterpret_cast<float *>(ring + G::R.pool + G::R.merge);
    float *sm = reinterpret_cast<float *>(ring + G::R.pool + G::R.merge + G::R.weights);   // [WARPS][8] maxima, then the CTA's
    float *sl = sm + (WARPS + MOST) * kBlock;                              // ... and sums
    __shared__ uint64_t full[kMaxRing], empty[kMaxRing];
    __shared__ uint8_t none[kMaxRing];
    __shared__ int part[32], start[2];
    __shared__ int gave_up, never;     // (gave_up: a hint to other waits that they need not run out too)
    __shared__ volatile int lost;      // tiles are missing: set by warps that compute, ahead of a barrier that all of them pass
    __shared__ long long place[MOST * kBlock];
    __shared__ float shares[kMaxCluster][MOST * kBlock];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // groups of a.blocks warps (the warps left over only help to join)
    const int group = warp / a.blocks, block = warp - group * a.blocks;
    const bool works = group < a.groups;
    if (tid == 0) {
        gave_up = never = 0;
        lost = 0;
        for (int s = 0; s < a.ring; ++s) {
            ptx::mbar_init(&full[s], 1);
            ptx::mbar_init(&empty[s], a.blocks);
        }
        ptx::fence_mbar_init();
        if (a.n_pages) {
            ptx::prefetch_tmap(&km);
            ptx::prefetch_tmap(&vm);
        }
    }
    kv4::after_the_kernel_before();

    // ---- this CTA's run
    Walk run{0, 0, 0, 0, 0, 0, 0, 0, 0};
    int rank = 0, cta = 0, total = 0, runs = 0;
    unsigned empty_seqs = 0;           // of up to 32
    bool any = false;
    if (a.cluster) {
        rank = (int)(blockIdx.x & (unsigned)(a.cluster - 1));
        const int unit = (int)(blockIdx.x >> a.cluster_log);
        run.b = a.by_units.into(unit);
        run.j = unit - run.b * units_of(a);
        run.set(a);
        if (tid == 0 && run.raw > capacity(a)) *a.status = GDN_ERR_PAGE;
        run.begin = run.n * rank >> a.cluster_log;     // (below 2^30: a length has 2^27 tiles at most)
        run.end = run.n * (rank + 1) >> a.cluster_log;
        any = run.begin < run.end;
        __syncthreads();
    } else {
        cta = (int)blockIdx.x;
        if (a.n_seqs <= 32) {          // each warp by itself, with one look at the lengths
            const int raw = lane < a.n_seqs ? max(a.lens[lane], 0) : 0;
            const int n = (min(raw, capacity(a)) + kTile - 1) / kTile, steps = steps_of(n) * units_of(a);
            if (warp == 0 && raw > capacity(a)) *a.status = GDN_ERR_PAGE;
            const int incl = warp_sum(steps, lane);
            total = __shfl_sync(0xffffffffu, incl, 31);
            runs = runs_of(a, total);
            const int from = cta < runs ? run_begin(total, runs, cta) : total;
            run.left = cta < runs ? run_begin(total, runs, cta + 1) - from : 0;
            const int src = __ffs(__ballot_sync(0xffffffffu, incl > from)) - 1;
            if (run.left > 0) {
                run.b = src;
                run.from = from - __shfl_sync(0xffffffffu, incl - steps, src);
                run.n = __shfl_sync(0xffffffffu, n, src);
                run.raw = __shfl_sync(0xffffffffu, raw, src);
            }
            empty_seqs = __ballot_sync(0xffffffffu, lane < a.n_seqs && n == 0);
            __syncthreads();
        } else {
            total = total_steps(a, part, G::ALL);
            runs = runs_of(a, total);
            const int from = cta < runs ? run_begin(total, runs, cta) : total;
            run.left = cta < runs ? run_begin(total, runs, cta + 1) - from : 0;
            if (warp == 0 && run.left > 0) {
                int before;
                const int b = find_step(a, from, lane, &before);
                if (lane == 0) {
                    start[0] = b;
                    start[1] = from - before;
                }
            }
            __syncthreads();
            if (run.left > 0) {
                run.b = start[0];
                run.from = start[1];
                run.set(a);
            }
        }
        if (run.left > 0) {
            run.j = run.from / steps_of(run.n);
            run.from -= run.j * steps_of(run.n);
            any = run.cut();
        }
        if (tid == 0 && gridDim.x > 1) open_of(a, gridDim.x, DV)[cta].parts = 0;
    }
    // ---- the last warps fill the ring with the run's tiles, each every kFillers-th of them (one alone would need
    // 700 cycles a tile, twice what HBM does)
    int s = 0;                         // a stage of the ring, and its phase
    uint32_t phase = 0;
    auto advance = [&](int by) {
        s += by;
        while (s >= a.ring) {
            s -= a.ring;
            phase ^= 1;
        }
        while (s < 0) {                // (a group whose last tiles in a segment were not there)
            s += a.ring;
            phase ^= 1;
        }
    };
    if (warp >= WARPS) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(G::FILL_REGS));
        const int who = warp - WARPS;  // stages who, who + kFillers, ...
        s = who;
        bool more = any && who < a.ring;
        int skip = who;                // of the segment's tiles, before this warp's first
        Walk w = run;
        while (more) {
            const int h = a.by_rb.into(w.j);
            int tile = w.begin + skip;
            while (more && tile < w.end) {
                // lane i: page of tile first + i, and that tile's first token in it
                const int first = tile;
                int page = -1, off = 0;
                if (first + lane < w.end) {
                    const int slot = a.by_tpp.into(first + lane);
                    page = a.table[(size_t)w.b * a.max_pages + slot];
                    off = (first + lane - slot * a.tpp) * kTile;
                }
                while (tile < first + 32 && tile < w.end) {
                    const int p = __shfl_sync(0xffffffffu, page, tile - first);
                    const int y = __shfl_sync(0xffffffffu, off, tile - first);
                    const bool came = ptx::mbar_wait(&empty[s], phase ^ 1, &gave_up);
                    if (__any_sync(0xffffffffu, !came)) {
                        gave_up = 1;
                        *a.status = GDN_ERR_TIMEOUT;
                        more = false;
                        break;
                    }
                    if (lane == 0) {
                        const bool there = (unsigned)p < (unsigned)a.n_pages;
                        none[s] = !there;
                        if (!there) {
                            *a.status = GDN_ERR_PAGE;
                            ptx::mbar_arrive(&full[s]);
                        } else {
                            ptx::mbar_arrive_expect_tx(&full[s], G::STAGE);
                            auto pick = [&](int x) { return (x & 3) == 0 ? y : (x & 3) == 1 ? h : p; };
                            uint8_t *stage = ring + s * G::STAGE;
                            const int k1 = pick(a.k_order), k2 = pick(a.k_order >> 2), k3 = pick(a.k_order >> 4);
#pragma unroll
                            for (int c = 0; c < G::KB / 2048; ++c)
                                ptx::tma_load_4d(stage + c * 2048, &km, &full[s], c * G::BOX, k1, k2, k3);
                            const int v1 = pick(a.v_order), v2 = pick(a.v_order >> 2), v3 = pick(a.v_order >> 4);
#pragma unroll
                            for (int c = 0; c < G::VB / 2048; ++c)
                                ptx::tma_load_4d(stage + G::KB + c * 2048, &vm, &full[s], c * G::BOX, v1, v2, v3);
                        }
                    }
                    // the next of this warp's stages, in this lap of the ring or the next
                    if (s + kFillers < a.ring) {
                        s += kFillers;
                        tile += kFillers;
                    } else {
                        tile += a.ring - s + who;
                        s = who;
                        phase ^= 1;
                    }
                }
            }
            skip = tile - w.end;       // tiles go on in order over the segments
            more = more && w.next(a);
        }
        // Copies land before the CTA can exit, whether those who wanted them still wait or gave up: the last use of each
        // of this warp's stages, in this lap or the one before.
        for (int i = who; i < a.ring; i += kFillers)
            if (!ptx::mbar_wait(&full[i], i < s ? phase : phase ^ 1, &never)) {
                *a.status = GDN_ERR_TIMEOUT;
                break;
            }
        if (a.cluster > 1) {
            cluster_sync();
            cluster_sync();
        }
        return;
    }
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(G::WORK_REGS));
    if (!a.cluster)                    // rows of empty sequences
        for (int b = cta; b < a.n_seqs; b += gridDim.x)
            if (a.n_seqs <= 32 ? empty_seqs >> b & 1 : tiles_at(a, b) == 0)
                for (int i = tid; i < a.n_q * a.H * (DV / 4); i += G::THREADS)
                    store4(a.out, a.out_type, (size_t)b * a.n_q * a.H * DV + 4 * (size_t)i, make_float4(0.f, 0.f, 0.f, 0.f));
    auto consumers_sync = [] { ptx::named_sync(1, G::THREADS); };

    // ---- segments
    float *pt = pts + (G::MMA16 ? 0 : warp * kBlock * 20);
    bool dead = false;
    auto row0_of = [&](const Walk &w) { return (w.j - a.by_rb.into(w.j) * a.n_rb) * a.blocks * kBlock; };
    uint32_t next_q[Part::MMA16 ? Part::KS : 1][2];    // the next segment's queries, loaded while this one's parts join
    if (any || a.cluster) Part::load_queries(a, run, row0_of(run) + block * kBlock, lane, next_q);
    if (works) advance(group);         // s: where the group's next tile comes
    for (bool more = any || a.cluster; more;) {
        const int hk = a.by_rb.into(run.j), row0 = row0_of(run);
        Part u;
        if constexpr (!G::MMA16) {
            Part::stage_queries(a, run.b, hk, row0, sq);
            consumers_sync();
        }
#pragma unroll
        for (int i = 0; i < (Part::MMA16 ? Part::KS : 1); ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) u.qf[i][e] = next_q[i][e];
        u.begin(a, run, row0 + block * kBlock, lane);
        int tile = run.begin + group;
        while (works && tile < run.end) {
            if (!dead) {
                dead = __any_sync(0xffffffffu, !ptx::mbar_wait(&full[s], phase, &gave_up));
                if (dead) {
                    gave_up = 1;
                    lost = 1;
                    *a.status = GDN_ERR_TIMEOUT;
                }
            }
            if (!dead) {
                if (!none[s])
                    u.tile(a, ring + s * G::STAGE, tile * kTile, sq + block * G::QBLOCK, pt, lane);
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&empty[s]);
            }
            advance(a.groups);
            tile += a.groups;
        }
        // to the group's first tile of the next segment: tiles go on in order
        if (works) advance(run.end - (tile - group));
        u.finish();
        Walk next = run;
        more = any && next.next(a);
        if (more) Part::load_queries(a, next, row0_of(next) + block * kBlock, lane, next_q);

        // ---- the groups' parts of the segment join: MC columns at a time, or, when no more tiles come, all of
        // them in the ring
        const int g = lane >> 2, t = lane & 3;
        const bool whole = run.begin == 0 && run.end == run.n, mine = works && !(COLS && t >= 2);
        const int rows = a.blocks * kBlock, valid = COLS ? 4 : rows;
        const bool final = whole && a.cluster < 2;
        float *part_out = whole || a.cluster ? nullptr
                                             : a.ws + partial_slot(cta, run.begin == 0) * partial_size(rows, DV);
        if (part_out && run.begin == 0 && tid == 0) {  // the runs up to that of the unit's last step go on with it
            const int end = run_begin(total, runs, cta + 1) + run.n + kUnitCost - run.to;
            open_of(a, gridDim.x, DV)[cta] = {run.b, run.j, run_of(total, runs, end - 1) - cta + 1, 0};
        }
        if (g == 0 && mine)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                sm[warp * kBlock + 2 * t + r] = u.m[r];
                sl[warp * kBlock + 2 * t + r] = u.l[r];
            }
        consumers_sync();               // (every group is done with the ring, too)
        // The same answer for all of them, whichever warp's wait it was that gave up: how many barriers follow goes by it.
        // Then copies into the ring may still be under way, and nobody waits for a stage any more: in the next segment it
        // could be another group's, which has not seen its last use end.
        dead = lost;
        const bool last = !more && !dead;
        const int width = last ? DV : G::MC, pitch = width + 4;
        float *parts = last ? reinterpret_cast<float *>(ring) : merge;
        if (last && tid == 0)          // the second kernel may be set up meanwhile (0.3 us)
            asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        // half a warp a row: the parts' factors in place of their maxima, 1 / sum among them where they make the output
        for (int row = tid >> 4; row < (valid + 1) / 2 * 2; row += G::THREADS / 16) {
            const int w = tid & 15;
            const float mw = w < a.groups && row < valid ? sm[w * rows + row] : -INFINITY;
            const float lw = w < a.groups && row < valid ? sl[w * rows + row] : 0.f;
            const float M = max16(mw);
            // (a part of NaN scores has no maximum: the row is NaN)
            const float f = lw == lw ? weight(mw, M) : lw, L = sum16(f * lw);
            if (row < valid) {
                if (w < a.groups) sm[w * rows + row] = !final ? f : L == 0.f ? 0.f : f * __frcp_rn(L);
                if (w == 15) place[row] = row0 + row < a.R ? out_row(a, run.b, hk, row0 + row) : -1;
                if (w == 0 && part_out) {
                    part_out[rows * DV + row] = M;
                    part_out[rows * (DV + 1) + row] = L;
                } else if (w == 0) {
                    sm[WARPS * kBlock + row] = M;
                    sl[WARPS * kBlock + row] = L;
                }
            }
        }
#pragma unroll
        for (int c0 = 0; c0 < DV; c0 += G::MC) {
            if (mine) {
                float *p = parts + (warp * kBlock + 2 * t) * pitch + Part::element_of(0, 0, g) + (last ? c0 : 0);
#pragma unroll
                for (int i = 0; i < G::MC / 16; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        p[(e & 1) * pitch + Part::element_of(i, e, 0)] = u.o[c0 / 16 + i][e];
            }
            if (last && c0 + G::MC < DV) continue;
            const int from = last ? 0 : c0;
            consumers_sync();
#pragma unroll 1
            for (int x = tid; x < valid * (width / 4); x += G::THREADS) {
                const int row = x / (width / 4), c = x - row * (width / 4);    // (a power of two)
                float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < WARPS; ++w)
                    if (w < a.groups)
                        y = fma4(sm[w * rows + row], *reinterpret_cast<const float4 *>(parts + (w * rows + row) * pitch + 4 * c), y);
                if (final) {
                    if (place[row] >= 0) store4(a.out, a.out_type, (size_t)place[row] * DV + from + 4 * c, y);
                } else if (part_out) {
                    *reinterpret_cast<float4 *>(part_out + row * DV + from + 4 * c) = y;
                } else {
                    *reinterpret_cast<float4 *>(parts + row * pitch + 4 * c) = y;
                }
            }
            if (!last) consumers_sync();
        }
        if (a.cluster > 1) {           // ... and the CTAs': each takes its share of the rows' elements
            cluster_sync();
            // (a CTA whose waits gave up has joined them elsewhere: the outputs are lost, the status says so)
            for (int row = tid >> 4; row < (valid + 1) / 2 * 2; row += G::THREADS / 16) {
                const int p = tid & 15;
                const bool there = p < a.cluster && row < valid;
                const float mp = there ? peer_float(sm + WARPS * kBlock + row, p) : -INFINITY;
                const float lp = there ? peer_float(sl + WARPS * kBlock + row, p) : 0.f;
                const float M = max16(mp);
                const float f = lp == lp ? weight(mp, M) : lp, L = sum16(f * lp);
                if (there) shares[p][row] = L == 0.f ? 0.f : f * __frcp_rn(L);
            }
            consumers_sync();
            for (int x = rank * G::THREADS + tid; x < valid * (DV / 4); x += a.cluster * G::THREADS) {
                const int row = x / (DV / 4), c = x - row * (DV / 4);
                float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                for (int p = 0; p < a.cluster; ++p)
                    y = fma4(shares[p][row], peer_float4(reinterpret_cast<float *>(ring) + row * (DV + 4) + 4 * c, p), y);
                if (place[row] >= 0) store4(a.out, a.out_type, (size_t)place[row] * DV + 4 * c, y);
            }
            cluster_sync();            // peers are done reading
        }
        run = next;
    }
}

// Joins the parts of units that runs cut: block (c, y) is for the unit that run c leaves open, and rows y, y +
// gridDim.y, ... of it.  Groups of threads take parts in turn, each with its own running maximum.
constexpr int kJoinThreads = 256;
template <int DV>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const Attn a, const int runs) {
    constexpr int COLS4 = DV / 4, GROUPS = kJoinThreads / COLS4;
    __shared__ float4 sums[kJoinThreads];
    __shared__ float tops[GROUPS], totals[GROUPS];
    kv4::after_the_kernel_before();
    const int c = (int)blockIdx.x, rows = a.blocks * kBlock;
    const Open open = open_of(a, runs, DV)[c];
    if (open.parts < 2) return;
    const int hk = a.by_rb.into(open.j), row0 = (open.j - hk * a.n_rb) * rows;
    const int group = threadIdx.x / COLS4, col = threadIdx.x - group * COLS4;
    for (int row = (int)blockIdx.y; row < rows && row0 + row < a.R; row += gridDim.y) {
        float M = -INFINITY, L = 0.f;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int p = group; p < open.parts; p += GROUPS) {
            // (the unit begins in run c: its part in that run's second place)
            const float *q = a.ws + partial_slot(c + p, p == 0) * partial_size(rows, DV);
            const float m = q[rows * DV + row], l = q[rows * (DV + 1) + row];
            const float4 x = *reinterpret_cast<const float4 *>(q + row * DV + 4 * col);
            const float top = fmaxf(M, m), g = weight(M, top), f = l == l ? weight(m, top) : l;
            M = top;
            L = fmaf(f, l, L * g);
            y = fma4(f, x, make_float4(y.x * g, y.y * g, y.z * g, y.w * g));
        }
        sums[threadIdx.x] = y;
        if (col == 0) {
            tops[group] = M;
            totals[group] = L;
        }
        __syncthreads();
        if (group == 0) {
#pragma unroll
            for (int k = 0; k < GROUPS; ++k) M = fmaxf(M, tops[k]);
            L = 0.f;
            y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < GROUPS; ++k) {
                const float f = totals[k] == totals[k] ? weight(tops[k], M) : totals[k];
                L = fmaf(f, totals[k], L);
                y = fma4(f, sums[k * COLS4 + col], y);
            }
            const float f = L == 0.f ? 0.f : __frcp_rn(L);
            store4(a.out, a.out_type, (size_t)out_row(a, open.b, hk, row0 + row) * DV + 4 * col,
                   make_float4(y.x * f, y.y * f, y.z * f, y.w * f));
        }
        __syncthreads();
    }
}

template <typename T, int DK, int DV, int WARPS, int MOST, bool COLS>
cudaError_t launch_one(const CUtensorMap &km, const CUtensorMap &vm, const Attn &a, int grid, cudaStream_t stream) {
    using G = Geo<T, DK, DV, WARPS, MOST>;
    static PerDeviceOnce setup;
    cudaError_t e = setup.run([] {
        cudaFuncAttributes f;
        const cudaError_t q = cudaFuncGetAttributes(&f, attn_kernel<T, DK, DV, WARPS, MOST, COLS>);
        if (q != cudaSuccess) return q;
        if (f.numRegs < G::REGS) return cudaErrorInvalidConfiguration;   // (the split counts on them)
        return cudaFuncSetAttribute(attn_kernel<T, DK, DV, WARPS, MOST, COLS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
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
    cfg.blockDim = dim3(G::ALL);
    cfg.dynamicSmemBytes = G::SMEM;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, attn_kernel<T, DK, DV, WARPS, MOST, COLS>, km, vm, a);
    if (e != cudaSuccess || a.cluster || grid < 2) return e;
    return kv4::launch_early(join_kernel<DV>, dim3((unsigned)grid - 1, (unsigned)(a.R < 8 ? a.R : 8)), kJoinThreads, 0, stream,
                             a, grid);
}

template <typename T, int DK, int DV>
cudaError_t launch_rows(const CUtensorMap &km, const CUtensorMap &vm, const Attn &a, int grid, cudaStream_t stream) {
    constexpr int E = (int)sizeof(T);
    constexpr Share few = share_of(DK, DV, E, 1), many = share_of(DK, DV, E, kBlock + 1);
    if constexpr (E == 4) {
        if (a.R <= kBlock) return launch_one<T, DK, DV, few.warps, few.most, false>(km, vm, a, grid, stream);
    } else {
        // of at most 4 rows, the weights' second terms enter in the free columns of the same MMAs
        if (a.R <= 4) return launch_one<T, DK, DV, few.warps, few.most, true>(km, vm, a, grid, stream);
    }
    return launch_one<T, DK, DV, many.warps, many.most, false>(km, vm, a, grid, stream);
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
