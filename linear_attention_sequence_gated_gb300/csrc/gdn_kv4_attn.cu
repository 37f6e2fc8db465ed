// Decode attention over the 4-bit cache (gdn_flash_attn_kv4): for every
// sequence b, query head h and query i,
//     out[b, i, h, :] = softmax_j(scale q[b,h,i] . k[b,hk,j] + mask[b,0,i,j]) v[b,hk,j,:]
// over the tokens j that the sequence holds (with `causal`, up to the query's
// own), hk = h / (n_heads / n_heads_kv), k and v as the cache keeps them.
//
// The cache is streamed once: 9/16 byte an element, so at 128 + 128 elements a
// token 144 bytes against 512 in bf16, and the question is whether the codes can
// be turned into MMA operands as fast as they arrive.  Decoding is exact (the
// values have 6 bits), so K and V enter f16 MMAs (m16n8k16, fp32 accumulators)
// without a rounding:
//     S^T  = K Q^T      M = 16 tokens (one tile), N = 8 rows, K = elements
//     O^T += V^T P^T    M = 16 elements, N = 8 rows, K = 16 tokens
// with rows = (query head of the group, query).  The contraction index of an MMA
// may be permuted as long as both operands agree, and so may the rows of M: the
// tile's order (gdn_kv4.cuh) is chosen so that a lane's codes are whole 16-byte
// words, one or two scales serve all of a lane's key codes, and one scale a token
// all of its value codes.  A pair of values costs one conversion
// and one multiplication.
//   * q is scaled to 2^14 by a power of two per row and held as f16: exact for
//     f16 and (all but elements 2^-28 of the row's largest) bf16 queries; fp32
//     queries take a second f16 for the remainder (22 bits).
//   * The probabilities, scaled by 2^12 to keep small ones out of f16's
//     subnormals, enter as hi + lo f16 (22 bits), transposed in registers by
//     movmatrix: lane (g, t) holds S^T of tokens g and rows 2t, 2t + 1 and needs
//     P^T of row g and tokens 2t, 2t + 1.
// Scores, maxima, sums and the output accumulate in fp32.
//
// Work is shared out in steps of 2 or 4 tiles, not in sequences: the steps of all
// (sequence, kv head, row block) units in a row are cut into equal runs, one a warp, so
// ragged batches and single long sequences load the GPU evenly.  A warp that has a unit
// to itself writes its output; otherwise it leaves (max, sum, output) in the
// workspace and a second kernel, launched as a programmatic dependent, joins the
// parts in a fixed order (results do not depend on timing).  It also writes the
// zero rows of empty sequences.  A call with few units of few tiles gives each unit
// a CTA instead, whose warps join their parts in shared memory: one launch.
#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/gdn.h"
#include "gdn_internal.h"
#include "gdn_kv4.cuh"
#include "gdn_ptx.cuh"

namespace gdn {
namespace kv4 {
namespace {

constexpr int kGrid = 152;             // CTAs: one per SM of the GPU this is written for (and what the
                                       // workspace's size goes by, on any device)

// Rows of a unit: one MMA column tile.  More rows of a kv head are more units, which
// decode the tiles again (from L2): blocks of 16 rows decode half as often, but took
// twice the registers and so half the warps, and 16 x 5 queries x 32/8 x 5001 x 128 took
// 57 us so and 49 us with blocks of 8.  (Steps of 128 tokens decoded once for 32 rows
// into operand tiles of tcgen05.mma took 99 us: the chain of copy, decoding, product,
// softmax and product across warps is 2.4 us a step and 8 us a unit.)
constexpr int kRows = 8;

// Shape of the kernel for widths DK and DV.  Each warp streams its run through a ring
// of its own in shared memory: stages of U tiles, each tile one bulk copy.  12 warps
// and steps of 4 tiles where 168 registers a thread hold the output tile and two
// steps' tiles (kColumns and kHi: 143 to 162 registers; kHiLo spills 20 to 80 bytes a
// thread there, with fp32 queries 24 to 136), else 8 and 2 (256 x 256 with fp32 queries
// spills 16).  (64 x 32/8 x 4096 x 128: 61 us; 12 warps with steps of 2 tiles 72, with
// steps of 3 68; 8 warps with steps of 4 82, 16 with steps of 2 72, both when it took
// 68.)
constexpr int warps_of(int dk, int dv) { return dk <= 128 && dv <= 128 ? 12 : 8; }
constexpr int step_of(int dk, int dv) { return warps_of(dk, dv) == 12 ? 4 : 2; }
template <int DK, int DV>
struct Geo {
    static constexpr int WARPS = warps_of(DK, DV);
    static constexpr int U = step_of(DK, DV);          // tiles of a step
    static constexpr int TB = tile_bytes(DK, DV);
    static constexpr int BUDGET = 216 * 1024;
    static constexpr int FIT = BUDGET / (WARPS * U * TB);
    static constexpr int STAGES = FIT < 8 ? FIT : 8;
    static constexpr int RING = STAGES * U * TB;       // of a warp
    static constexpr int SMEM = WARPS * RING;
    static_assert(STAGES >= 2 && TB % 16 == 0, "ring");
};

struct Attn {
    View c;
    const void *q, *mask;
    void *out;
    float *ws;
    int n_seqs, H, n_q, R, n_rb, W;    // R rows a kv head in n_rb blocks; W runs at most
    float scale;
    int q_type, out_type;
    bool causal;
    bool alone;                        // a block a unit, and no partial results
};

// How the weights enter the MMAs.  kHi: 11 bits, for 16-bit outputs of 16-bit queries,
// whose own rounding is as large or larger: over 60 shapes the error against 64 bits is
// 1.00 to 1.01 of what that rounding alone makes for bf16, 1.00 to 1.37 for f16.  (22
// bits cost 0.3 to 0.5 us a call with kColumns.)  kHiLo: the remainder's 11 bits in a
// second MMA.  kColumns: of at most 4 rows, the remainder
// in the other 4 columns of the same MMA, where row r's queries stand again as
// column r + 4; the two columns' outputs are added at the end.
enum Weights { kHi = 0, kHiLo = 1, kColumns = 2 };

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kPBits = 12.f;         // probabilities are scaled by 2^12
constexpr float kFar = 65536.f;        // scores from which weights go by differences (fp32's unit: 2^-7)
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// the same with a zero accumulator
__device__ __forceinline__ void mma0(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// 8 x 8 transpose of 16-bit elements across the warp: lane (g, t) gives row g,
// columns 2t, 2t + 1 and gets row g of the transpose.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t half2_bits(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
// (x, y) as f16 pairs hi + lo
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) {
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    hi = half2_bits(h);
    lo = half2_bits(__floats2half2_rn(x - f.x, y - f.y));
}

__device__ __forceinline__ float element(const void *p, int type, size_t i) {
    if (type == GDN_DTYPE_F32) return static_cast<const float *>(p)[i];
    const unsigned short u = static_cast<const unsigned short *>(p)[i];
    return type == GDN_DTYPE_BF16 ? __uint_as_float((uint32_t)u << 16) : __half2float(__ushort_as_half(u));
}

// 8 consecutive outputs
__device__ __forceinline__ void store8(void *out, int type, size_t i, const float (&x)[8]) {
    if (type == GDN_DTYPE_F32) {
        float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(out) + i);
        p[0] = make_float4(x[0], x[1], x[2], x[3]);
        p[1] = make_float4(x[4], x[5], x[6], x[7]);
        return;
    }
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (type == GDN_DTYPE_BF16) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
            w[e] = *reinterpret_cast<const uint32_t *>(&h);
        } else {
            w[e] = half2_bits(__floats2half2_rn(x[2 * e], x[2 * e + 1]));
        }
    }
    *reinterpret_cast<uint4 *>(static_cast<unsigned short *>(out) + i) = make_uint4(w[0], w[1], w[2], w[3]);
}

// 2 consecutive outputs
__device__ __forceinline__ void store2(void *out, int type, size_t i, float x, float y) {
    if (type == GDN_DTYPE_F32)
        *reinterpret_cast<float2 *>(static_cast<float *>(out) + i) = make_float2(x, y);
    else if (type == GDN_DTYPE_BF16)
        *reinterpret_cast<__nv_bfloat162 *>(static_cast<__nv_bfloat16 *>(out) + i) = __floats2bfloat162_rn(x, y);
    else
        *reinterpret_cast<__half2 *>(static_cast<__half *>(out) + i) = __floats2half2_rn(x, y);
}

__device__ __forceinline__ int tiles_of(int len) { return (len + kTile - 1) / kTile; }

// Steps of U tiles are counted from each unit's start and never cut, since a step of
// fewer tiles takes as long (8 x 8 kv heads x 3000 x 128: 16.0 us, and 19.1 with runs of
// equal tiles).
__device__ __forceinline__ int steps_of(int tiles, int U) { return (tiles + U - 1) / U; }

// Runs of a call of T steps: of at least 4 tiles, which a warp decodes in about the time
// that it waits for one, and the fewer parts there are to join (1 sequence x 20000 tokens:
// 24.6 us with runs of 1 tile and more, 16.9 of 2, 12.9 of 4).
__device__ __forceinline__ int runs_of(const Attn &a, int T, int U) { return min(a.W, steps_of(T, 4 / U)); }

// Tiles of a unit of sequence b.
__device__ __forceinline__ int tiles_at(const Attn &a, int b) {
    if (b >= a.n_seqs) return 0;
    const int raw = a.c.lens[b];
    if (raw > capacity(a.c)) *a.c.status = GDN_ERR_PAGE;
    return tiles_of(min(max(raw, 0), capacity(a.c)));
}
// Whole-warp: the steps of all units of the sequences from `b0` to before `end`, and the
// sequence that step x lies in with the steps before it.
__device__ __forceinline__ int steps_between(const Attn &a, int U, int units, int b0, int end, int lane) {
    int n = 0;
#pragma unroll 4
    for (int b = b0 + lane; b < end; b += 32) n += steps_of(tiles_at(a, b), U) * units;
    return __reduce_add_sync(0xffffffffu, n);
}
__device__ __forceinline__ int find_step(const Attn &a, int U, int units, int x, int lane, int *before) {
    int done = 0;
    for (int base = 0;; base += 32) {
        const int n = steps_of(tiles_at(a, base + lane), U) * units;
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

// A partial result: [rows][DV] outputs, [rows] maxima, [rows] sums.
template <int DV> constexpr size_t kPartial = (size_t)kRows * (DV + 2);

// One warp's share of one unit: an online softmax over tiles.
template <int DK, int DV, bool QLO, int PM>
struct Unit {
    static constexpr int U = Geo<DK, DV>::U, TB = tile_bytes(DK, DV);
    static constexpr int CK = DK > 128 ? 2 : 1;        // key parts
    static constexpr int ST = DK >= 128 ? 8 : 4;       // MMA steps of a part
    static constexpr int VB = DV / 64;                 // value blocks, four M tiles each
    uint32_t qh[CK * ST][2], ql[QLO ? CK * ST : 1][2];
    float f[2];                        // row factors of the scores (not negative)
    int qi[2];                         // the row's query; -1: no such row
    int all;                           // tokens that every row sees and no mask changes
    float m[2], l[2];                  // running maximum, sum of the weights
    float o[VB * 4][4];

    __device__ __forceinline__ void begin(const Attn &a, int b, int hk, int rb, int lane) {
        const int g = lane >> 2, t = lane & 3;
        const int rep = a.H / a.c.Hkv;
        const int raw = max(a.c.lens[b], 0), len = min(raw, capacity(a.c));
        all = a.mask ? 0 : (a.causal ? min(len, max(raw - a.n_q + 1, 0)) : len);
        // all loads first: a lane's elements are whole 16-byte words
        constexpr int QE = QLO ? 4 : 8, QW = ST * 4 / QE;   // elements a word, words a part
        uint4 raw_q[CK][QW];
        const int row = PM == kColumns ? g & 3 : rb * kRows + g;
        const size_t q0 = ((size_t)(b * (size_t)a.H + hk * rep) * a.n_q + row) * DK;
        const uint4 *at = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(a.q) +
                                                          (q0 + t * ST * 4) * (16 / QE));
#pragma unroll
        for (int c = 0; c < CK; ++c)
#pragma unroll
            for (int i = 0; i < QW; ++i)
                raw_q[c][i] = row < a.R ? at[c * (128 / QE) + i] : make_uint4(0, 0, 0, 0);
        float x[CK * ST * 4];
        float big = 0.f;
#pragma unroll
        for (int c = 0; c < CK; ++c)
#pragma unroll
            for (int i = 0; i < QW; ++i) {
                const uint32_t w[4] = {raw_q[c][i].x, raw_q[c][i].y, raw_q[c][i].z,
                                       raw_q[c][i].w};
                float *y = x + (c * QW + i) * QE;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if constexpr (QLO) {
                        y[e] = __uint_as_float(w[e]);
                    } else if (a.q_type == GDN_DTYPE_BF16) {
                        y[2 * e] = __uint_as_float(w[e] << 16);
                        y[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
                    } else {
                        const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&w[e]));
                        y[2 * e] = h.x;
                        y[2 * e + 1] = h.y;
                    }
                }
            }
#pragma unroll
        for (int e = 0; e < CK * ST * 4; ++e) big = fmaxf(big, fabsf(x[e]));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
        // 2^14 / (the power of two at or below the row's largest element)
        // (from 2^-112 down the factor stays 2^126, with which the least fp32 number, 2^-149,
        // is still two units of f16's subnormals)
        const int ex = min(max((int)(__float_as_uint(big) >> 23) - 127, -112), 127);
        const float up = __uint_as_float((uint32_t)(14 - ex + 127) << 23);
        const float back = __uint_as_float((uint32_t)(ex - 14 + 127) << 23) * fabsf(a.scale);
        const float sup = a.scale < 0.f ? -up : up;   // q takes the scale's sign
#pragma unroll
        for (int s = 0; s < CK * ST; ++s)
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const float x0 = x[s * 4 + 2 * p] * sup, x1 = x[s * 4 + 2 * p + 1] * sup;
                if constexpr (QLO) split2(x0, x1, qh[s][p], ql[s][p]);
                else qh[s][p] = half2_bits(__floats2half2_rn(x0, x1));
            }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            f[r] = __shfl_sync(0xffffffffu, back, (2 * t + r) * 4);
            const int mine = PM == kColumns ? (2 * t + r) & 3 : rb * kRows + 2 * t + r;
            qi[r] = mine < a.R ? mine % a.n_q : -1;
            m[r] = -INFINITY;
            l[r] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < VB * 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    }

    // U tiles at `p`, tokens pos .. of a sequence; from `stop` on they are not this
    // warp's or not there, and tile i counts only if bit i of `good` is set.
    __device__ __forceinline__ void tiles(const Attn &a, const uint8_t *p, int b, int pos, int stop, unsigned good,
                                          int lane) {
        const int g = lane >> 2, t = lane & 3;
        const int ka = 4 * (g >> 1) + (g & 1), kb = ka + 2;   // tokens of C rows g, g + 8
        float s[U][4];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint8_t *k = p + u * TB;
#pragma unroll
            for (int c = 0; c < CK; ++c) {
                uint32_t wa[ST / 2], wb[ST / 2];       // two steps' codes a word
                uint32_t sa, sb;                       // f16 scales of the lane's one or two groups
                if constexpr (ST == 8) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(k + c * 1024 + ka * 64 + t * 16);
                    const uint4 y = *reinterpret_cast<const uint4 *>(k + c * 1024 + kb * 64 + t * 16);
                    wa[0] = x.x; wa[1] = x.y; wa[2] = x.z; wa[3] = x.w;
                    wb[0] = y.x; wb[1] = y.y; wb[2] = y.z; wb[3] = y.w;
                    const uint8_t *sc = k + 8 * DK + c * 128 + 2 * t;
                    sa = scales01(*reinterpret_cast<const uint16_t *>(sc + ka * 8));
                    sb = scales01(*reinterpret_cast<const uint16_t *>(sc + kb * 8));
                } else {
                    const uint2 x = *reinterpret_cast<const uint2 *>(k + ka * 32 + t * 8);
                    const uint2 y = *reinterpret_cast<const uint2 *>(k + kb * 32 + t * 8);
                    wa[0] = x.x; wa[1] = x.y;
                    wb[0] = y.x; wb[1] = y.y;
                    const uint8_t *sc = k + 8 * DK + t;
                    sa = scales01(sc[ka * 4]);
                    sb = scales01(sc[kb * 4]);
                }
#pragma unroll
                for (int h = 0; h < ST / 2; ++h) {
                    uint32_t x[4], y[4];
                    decode4(wa[h], x);
                    decode4(wb[h], y);
                    const bool second = ST == 8 && h >= 2;
                    const uint32_t da = second ? dup_hi(sa) : dup_lo(sa), db = second ? dup_hi(sb) : dup_lo(sb);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t A[4] = {mul2(x[2 * i], da), mul2(y[2 * i], db), mul2(x[2 * i + 1], da),
                                               mul2(y[2 * i + 1], db)};
                        const int st = c * ST + 2 * h + i;
                        if (st == 0) mma0(s[u], A, qh[st][0], qh[st][1]);
                        else mma(s[u], A, qh[st][0], qh[st][1]);
                        if constexpr (QLO) mma(s[u], A, ql[st][0], ql[st][1]);
                    }
                }
            }
        }
        const bool plain = pos + U * kTile <= min(all, stop) && good == (1u << U) - 1u;
        uint32_t ph[U][2], pl[PM == kHiLo ? U : 1][2];
        float cf[2];
        if (!plain) {
            const int raw = max(a.c.lens[b], 0);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                // (a length past the table counts in full for the causal limit)
                const int i = qi[r];
                const int lim = a.causal ? (int)min((long long)stop, (long long)raw - a.n_q + 1 + i) : stop;
                const size_t row = ((size_t)b * a.n_q + i) * (size_t)capacity(a.c);
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int e = r; e < 4; e += 2) {
                        const int key = pos + u * kTile + (e < 2 ? ka : kb);
                        float x = s[u][e] * f[r];
                        if (i < 0 || key >= lim || !(good >> u & 1)) x = -INFINITY;
                        else if (a.mask) x += element(a.mask, a.q_type, row + key);
                        s[u][e] = x;
                    }
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float mx = fmaxf(s[0][r], s[0][r + 2]);
#pragma unroll
            for (int u = 1; u < U; ++u) mx = fmaxf(mx, fmaxf(s[u][r], s[u][r + 2]));
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            // The weight of a score x is 2^((x - maximum) log2 e + 12).  Without a
            // mask that is one FMA on the MMAs' result and the maximum's rounded
            // product; the factor for what earlier steps summed takes the difference
            // of two such products, each rounded by itself (not contracted into an
            // FMA), so it is exactly 1 while the maximum stands: a residue of one
            // rounding there would scale the older tokens again at every step of a run
            // (512 steps, scores near 40: outputs off by 1.6e-3 of their RMS, 9e-5
            // at most without it).  Scores that took a mask are differences in natural units
            // first: masks of the type's lowest value would overflow.  So are scores
            // beside a maximum of kFar and more, where the product's rounding would move
            // all weights together, at 1e7 out of f16's range.  A step in part without a
            // mask takes differences too, which is one rounding of the product apart from
            // the others (2^-24 of the score), as parts of different maxima are in the
            // join.
            const float old = m[r], mn = fmaxf(old, plain ? mx * f[r] : mx);
            m[r] = mn;
            const float base = mn == -INFINITY ? 0.f : mn;
            const bool far = !(fabsf(base) < kFar);
            cf[r] = exp2_approx(a.mask || far ? (old - base) * kLog2e
                                              : __fsub_rn(__fmul_rn(old, kLog2e), __fmul_rn(base, kLog2e)));
            float sum = 0.f;
            if (plain && !far) {
                const float k = f[r] * kLog2e, z = kPBits - __fmul_rn(base, kLog2e);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    s[u][r] = exp2_approx(fmaf(s[u][r], k, z));
                    s[u][r + 2] = exp2_approx(fmaf(s[u][r + 2], k, z));
                }
            } else {
                if (plain) {           // (the others took their factor above)
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        s[u][r] = __fmul_rn(s[u][r], f[r]);
                        s[u][r + 2] = __fmul_rn(s[u][r + 2], f[r]);
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    s[u][r] = exp2_approx(fmaf(__fsub_rn(s[u][r], base), kLog2e, kPBits));
                    s[u][r + 2] = exp2_approx(fmaf(__fsub_rn(s[u][r + 2], base), kLog2e, kPBits));
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) sum += s[u][r] + s[u][r + 2];
            l[r] = fmaf(l[r], cf[r], sum);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float x = s[u][2 * k], y = s[u][2 * k + 1];
                if constexpr (PM == kHi) {
                    ph[u][k] = half2_bits(__floats2half2_rn(x, y));
                } else if constexpr (PM == kHiLo) {
                    split2(x, y, ph[u][k], pl[u][k]);
                    pl[u][k] = transpose8(pl[u][k]);
                } else {
                    uint32_t lo;
                    split2(x, y, ph[u][k], lo);
                    if (t >= 2) ph[u][k] = lo;
                }
                ph[u][k] = transpose8(ph[u][k]);
            }
        // The products of U tiles add up in the MMAs, small terms first, and reach
        // the output by one fp32 FMA that also rescales it: the MMAs' accumulation
        // truncates, and over thousands of tokens that would show.
#pragma unroll
        for (int r = 0; r < VB; ++r) {
            uint32_t w[U][4], s01[U], s23[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint8_t *v = p + u * TB + 9 * DK;
                const uint4 x = *reinterpret_cast<const uint4 *>(v + ((r * 8 + g) * 4 + t) * 16);
                w[u][0] = x.x; w[u][1] = x.y; w[u][2] = x.z; w[u][3] = x.w;
                const int group = DV == 64 ? g >> 1 : (r >> 1) * 8 + g;
                uint32_t sw = *reinterpret_cast<const uint32_t *>(v + 8 * DV + group * 16 + 4 * t);
                // tokens that are not there: their scale bytes may hold anything, and
                // 0 times infinity would spoil the row
                if (!plain) {
                    const int left = (good >> u & 1) ? stop - (pos + u * kTile + 4 * t) : 0;
                    sw &= left >= 4 ? 0xffffffffu : (left <= 0 ? 0u : (1u << (8 * left)) - 1u);
                }
                s01[u] = scales01(sw);
                s23[u] = scales23(sw);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t A[U][4];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    uint32_t x[4];
                    decode4(w[u][i], x);
                    A[u][0] = mul2(x[0], s01[u]); A[u][1] = mul2(x[1], s01[u]);
                    A[u][2] = mul2(x[2], s23[u]); A[u][3] = mul2(x[3], s23[u]);
                }
                float d[4];
                if constexpr (PM == kHiLo) {
                    mma0(d, A[0], pl[0][0], pl[0][1]);
#pragma unroll
                    for (int u = 1; u < U; ++u) mma(d, A[u], pl[u][0], pl[u][1]);
                    mma(d, A[0], ph[0][0], ph[0][1]);
                } else {
                    mma0(d, A[0], ph[0][0], ph[0][1]);
                }
#pragma unroll
                for (int u = 1; u < U; ++u) mma(d, A[u], ph[u][0], ph[u][1]);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o[r * 4 + i][e] = fmaf(o[r * 4 + i][e], cf[e & 1], d[e]);
            }
        }
    }

    // The unit's rows: outputs where this warp saw all of its tiles, else a partial.
    __device__ __forceinline__ void end(const Attn &a, int b, int hk, int rb, bool whole, float *part, int lane) {
        const int g = lane >> 2, t = lane & 3, rep = a.H / a.c.Hkv;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float sum = l[r];
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            const int local = 2 * t + r, row = rb * kRows + local;
            if constexpr (PM == kColumns) {
#pragma unroll
                for (int i = 0; i < VB * 4; ++i) {
                    o[i][r] += __shfl_xor_sync(0xffffffffu, o[i][r], 2);
                    o[i][r + 2] += __shfl_xor_sync(0xffffffffu, o[i][r + 2], 2);
                }
            }
            if (row >= a.R) continue;
            const float inv = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
            const size_t at = (((size_t)b * a.n_q + row % a.n_q) * a.H + hk * rep + row / a.n_q) * DV;
#pragma unroll
            for (int blk = 0; blk < VB; ++blk) {
                const int el = 128 * (blk >> 1) + (DV == 64 ? 8 : 16) * g + 8 * (blk & 1);
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = o[blk * 4 + e / 2][2 * (e & 1) + r] * inv;
                if (whole) store8(a.out, a.out_type, at + el, x);
                else store8(part, GDN_DTYPE_F32, (size_t)local * DV + el, x);
            }
            if (!whole && g == 0) {
                part[kRows * DV + local] = m[r];
                part[kRows * (DV + 1) + local] = sum;
            }
        }
    }
};

// A walk over a run: the unit and the tile that it has reached.
template <int U>
struct Cursor {
    int left;                          // steps of the run from here on
    int b, u, j, n, len;               // sequence, unit of it, tile of the unit, tiles of a unit, tokens
    // the run's tiles of this unit
    __device__ __forceinline__ int tiles() const { return min(n - j, left * U); }
    // k tiles on (whole steps, or to the unit's end)
    __device__ __forceinline__ void next(const Attn &a, int units, int k) {
        left -= steps_of(k, U);
        j += k;
        if (j < n) return;
        j = 0;
        if (++u == units) {
            u = 0;
            if (left > 0) {            // the next sequence that holds anything
                do {
                    len = length(a.c, ++b);
                    n = tiles_of(len);
                } while (n == 0);
            }
        }
    }
};

template <int DK, int DV, bool QLO, int PM>
__global__ void __launch_bounds__(Geo<DK, DV>::WARPS * 32, 1) attn_kernel(const Attn a) {
    using G = Geo<DK, DV>;
    constexpr int U = G::U, ST = G::STAGES;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t full[G::WARPS][ST];
    __shared__ unsigned good[G::WARPS][ST];            // tiles of the stage whose pages exist
    __shared__ int steps[G::WARPS];
    __shared__ int gave_up;                            // (a hint only: other waits need not run out too)
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) gave_up = 0;
    if (lane < ST) {
        ptx::mbar_init(&full[warp][lane], 1);
        ptx::fence_mbar_init();        // (orders this lane's own barrier before the copies that signal it)
    }
    __syncthreads();
    after_the_kernel_before();
    const int units = a.c.Hkv * a.n_rb;
    Cursor<U> c;
    int w = 0, parts = 0;                              // this run's number; runs of the block's own unit
    if (a.alone) {
        c.b = blockIdx.x / units;
        c.u = blockIdx.x - c.b * units;
        c.len = length(a.c, c.b);
        const int n = tiles_at(a, c.b);
        parts = min(G::WARPS, n);
        c.j = warp < parts ? run_begin(n, parts, warp) : 0;
        c.n = warp < parts ? run_begin(n, parts, warp + 1) : 0;
        c.left = steps_of(c.n - c.j, U);
    } else {
        // the call's steps: the block scans the lengths together
        int T = 0;
        for (int b = threadIdx.x; b < a.n_seqs; b += G::WARPS * 32) T += steps_of(tiles_at(a, b), U) * units;
        T = __reduce_add_sync(0xffffffffu, T);
        if (lane == 0) steps[warp] = T;
        __syncthreads();
        T = 0;
#pragma unroll
        for (int k = 0; k < G::WARPS; ++k) T += steps[k];
        const int W = runs_of(a, T, U);
        // neighbouring runs on different SMs: few tiles spread over the GPU
        w = warp * gridDim.x + blockIdx.x;
        if (w >= W) return;
        const int at = run_begin(T, W, w);
        int before;
        c.left = run_begin(T, W, w + 1) - at;
        c.b = find_step(a, U, units, at, lane, &before);
        c.len = length(a.c, c.b);
        c.n = tiles_of(c.len);
        const int each = steps_of(c.n, U);
        c.u = (at - before) / each;
        c.j = (at - before - c.u * each) * U;
    }

    uint8_t *ring = smem + warp * G::RING;
    // Copies run ST - 1 stages ahead.  The tiles' addresses are looked up for a
    // window of up to 32 tiles of a unit at once, one a lane.
    Cursor<U> ahead = c;
    const uint8_t *src = nullptr;
    unsigned have = 0;                                 // tiles of the window whose pages exist
    int off = 0, count = 0, put = 0;                   // window's tiles copied, its tiles; next stage
    auto copy = [&]() {
        if (off == count) {
            if (ahead.left <= 0) return;
            off = 0;
            count = min(32, ahead.tiles());
            src = lane < count ? tile_ptr(a.c, ahead.b, ahead.u / a.n_rb, ahead.j + lane) : nullptr;
            have = __ballot_sync(0xffffffffu, src != nullptr);
            ahead.next(a, units, count);
        }
        const int k = min(U, count - off);
        const unsigned mine = have >> off & ((1u << k) - 1u);
        if (lane == 0) {
            good[warp][put] = mine;
            ptx::mbar_arrive_expect_tx(&full[warp][put], __popc(mine) * G::TB);
        }
        __syncwarp();
        if (lane >= off && lane < off + k && src)
            ptx::bulk_load(ring + (put * U + lane - off) * G::TB, src, G::TB, &full[warp][put]);
        off += k;
        put = put + 1 == ST ? 0 : put + 1;
    };
#pragma unroll 1
    for (int i = 0; i < ST - 1; ++i) copy();

    Unit<DK, DV, QLO, PM> unit;
    int get = 0;                                       // stage to read, and its barrier's phase
    uint32_t phase = 0;
    while (c.left > 0) {
        const int b = c.b, hk = c.u / a.n_rb, rb = c.u - hk * a.n_rb, j0 = c.j;
        const int j1 = c.j + c.tiles(), stop = min(c.len, j1 * kTile);
        unit.begin(a, b, hk, rb, lane);
        for (int j = j0; j < j1; j += U) {
            copy();                                    // into the stage that the last step left
            // (one answer for the warp: its lanes stay together whatever happens)
            if (!__all_sync(0xffffffffu, ptx::mbar_wait(&full[warp][get], phase, &gave_up))) {
                *a.c.status = GDN_ERR_TIMEOUT;
                gave_up = 1;
                // the copies in flight still write this block's shared memory
                const int never = 0;
                do {
                    ptx::mbar_wait(&full[warp][get], phase, &never, 1 << 28);
                    get = get + 1 == ST ? 0 : get + 1;
                    phase ^= get == 0;
                } while (get != put);
                c.left = 0;
                break;
            }
            unit.tiles(a, ring + get * U * G::TB, b, j * kTile, stop, good[warp][get], lane);
            __syncwarp();                              // the stage is read
            get = get + 1 == ST ? 0 : get + 1;
            phase ^= get == 0;
        }
        if (a.alone) break;
        const bool whole = j0 == 0 && j1 == c.n;
        unit.end(a, b, hk, rb, whole, a.ws + (size_t)partial_slot(w, j0 == 0) * kPartial<DV>, lane);
        c.next(a, units, j1 - j0);
    }
    if (!a.alone) return;

    // The block's own unit: its warps' parts meet in the rings' shared memory.
    __syncthreads();
    const int b = blockIdx.x / units, u = blockIdx.x - b * units, hk = u / a.n_rb, rb = u - hk * a.n_rb;
    float *part = reinterpret_cast<float *>(smem);
    if (warp < parts) unit.end(a, b, hk, rb, parts == 1, part + warp * kPartial<DV>, lane);
    if (parts == 1) return;
    __syncthreads();
    const int n_rows = min(kRows, a.R - rb * kRows);
    for (int i = threadIdx.x; i < n_rows * (DV / 4); i += G::WARPS * 32) {
        const int local = i / (DV / 4), x = i - local * (DV / 4), row = rb * kRows + local;
        const float *m = part + kRows * DV + local, *l = m + kRows;
        float top = -INFINITY, sum = 0.f;
        for (int k = 0; k < parts; ++k) top = fmaxf(top, m[k * kPartial<DV>]);
        const float base = top == -INFINITY ? 0.f : top;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < parts; ++k) {
            const float wt = exp2_approx((m[k * kPartial<DV>] - base) * kLog2e);
            const float4 v = reinterpret_cast<const float4 *>(part + k * kPartial<DV> + local * DV)[x];
            sum = fmaf(l[k * kPartial<DV>], wt, sum);
            y = make_float4(fmaf(v.x, wt, y.x), fmaf(v.y, wt, y.y), fmaf(v.z, wt, y.z), fmaf(v.w, wt, y.w));
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const size_t at = (((size_t)b * a.n_q + row % a.n_q) * a.H + hk * (a.H / a.c.Hkv) + row / a.n_q) * DV + 4 * x;
        store2(a.out, a.out_type, at, y.x * inv, y.y * inv);
        store2(a.out, a.out_type, at + 2, y.z * inv, y.w * inv);
    }
}

// Joins the partial results of the rows that several runs share.  A block has
// `rpb` rows, a warp each.  A warp reads the maxima and sums of up to 32 parts at
// once, so their weights are known before the outputs are read, and those loads
// do not wait for one another.  A row of more parts than a warp should take is left
// to the whole block, of JW warps: 16 where units have 128 parts and more (60000 tokens
// over one kv head: 15.7 us, and 19.2 with 8 warps; 63 parts of 3 x 2 kv heads at
// (64, 256): 14.1 and 13.4).
template <int DV>
struct Join {
    static constexpr int V = DV == 64 ? 2 : 4, C = DV == 256 ? 2 : 1;   // columns of a lane: C times V
    float x[C * V];
    float M, L;
    // parts first, first + step, ... below n of a row; part 0 is in its run's slot 1
    __device__ __forceinline__ void parts(const float *ws, int w0, int n, int local, int first, int step, int lane) {
        M = -INFINITY;
        L = 0.f;
#pragma unroll
        for (int e = 0; e < C * V; ++e) x[e] = 0.f;
        for (int p0 = first; p0 < n; p0 += 32 * step) {
            const int mine = p0 + lane * step, cnt = min(32, (n - p0 + step - 1) / step);
            const float *at = ws + (size_t)partial_slot(w0 + mine, mine == 0) * kPartial<DV>;
            float m = -INFINITY, l = 0.f;
            if (mine < n) {
                m = at[kRows * DV + local];
                l = at[kRows * (DV + 1) + local];
            }
            float top = m;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            top = fmaxf(top, M);
            const float base = top == -INFINITY ? 0.f : top;
            const float old = exp2_approx((M - base) * kLog2e), wt = exp2_approx((m - base) * kLog2e);
            M = top;
            float sum = l * wt;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            L = fmaf(L, old, sum);
#pragma unroll
            for (int e = 0; e < C * V; ++e) x[e] *= old;
            constexpr int B = 8;                       // loads in flight (they do not pass the shuffles)
            for (int i0 = 0; i0 < cnt; i0 += B) {
                float v[B][C * V];
#pragma unroll
                for (int i = 0; i < B; ++i) {
                    const int p = p0 + min(i0 + i, cnt - 1) * step;
                    const float *row = ws + (size_t)partial_slot(w0 + p, p == 0) * kPartial<DV> + local * DV;
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        if constexpr (V == 2) {
                            const float2 y = reinterpret_cast<const float2 *>(row)[lane];
                            v[i][0] = y.x; v[i][1] = y.y;
                        } else {
                            const float4 y = reinterpret_cast<const float4 *>(row + 128 * c)[lane];
                            v[i][4 * c] = y.x; v[i][4 * c + 1] = y.y; v[i][4 * c + 2] = y.z; v[i][4 * c + 3] = y.w;
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < B; ++i) {
                    const float k = __shfl_sync(0xffffffffu, wt, min(i0 + i, 31));
#pragma unroll
                    for (int e = 0; e < C * V; ++e)
                        if (i0 + i < cnt) x[e] = fmaf(v[i][e], k, x[e]);
                }
            }
        }
    }
    __device__ __forceinline__ int column(int c, int e, int lane) const { return c * 128 + lane * V + e; }
    __device__ __forceinline__ void store(const Attn &a, size_t at, int lane) const {
        const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int e = 0; e < V; e += 2) {
                store2(a.out, a.out_type, at + column(c, e, lane), x[c * V + e] * inv, x[c * V + e + 1] * inv);
            }
    }
};

template <int DV, int JW>
__global__ void __launch_bounds__(JW * 32) join_kernel(const Attn a, int U, int rpb, int n_rows) {
    __shared__ int s_w0[JW], s_n[JW];
    __shared__ float s_m[JW], s_l[JW], s_x[JW][DV];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int units = a.c.Hkv * a.n_rb;
    // the call's steps, and those before the block's first row's sequence: the block scans
    // the lengths together
    const int r0 = blockIdx.x * rpb, r = r0 + warp, b0 = r0 / a.R / a.c.Hkv;
    int all = 0, pre = 0;
    for (int b = threadIdx.x; b < a.n_seqs; b += JW * 32) {
        const int n = steps_of(tiles_at(a, b), U) * units;
        all += n;
        if (b < b0) pre += n;
    }
    all = __reduce_add_sync(0xffffffffu, all);
    pre = __reduce_add_sync(0xffffffffu, pre);
    if (lane == 0) {
        s_w0[warp] = all;
        s_n[warp] = pre;
    }
    __syncthreads();
    int T = 0, before = 0;
#pragma unroll
    for (int k = 0; k < JW; ++k) {
        T += s_w0[k];
        before += s_n[k];
    }
    __syncthreads();
    const int W = runs_of(a, T, U);
    auto place = [&](int r, int &local) {              // where a row's output goes
        const int unit = r / a.R, row = r - unit * a.R, b = unit / a.c.Hkv, hk = unit - b * a.c.Hkv;
        local = row % kRows;
        return (((size_t)b * a.n_q + row % a.n_q) * a.H + hk * (a.H / a.c.Hkv) + row / a.n_q) * DV;
    };
    int w0 = 0, n = -1;                                // runs that share the row; -1: none of ours
    if (warp < rpb && r < n_rows) {
        const int unit = r / a.R, row = r - unit * a.R, b = unit / a.c.Hkv, hk = unit - b * a.c.Hkv;
        const int steps = steps_of(tiles_of(length(a.c, b)), U);
        n = 0;
        if (steps > 0) {
            const int first = before + steps_between(a, U, units, b0, b, lane) + (hk * a.n_rb + row / kRows) * steps;
            w0 = run_of(T, W, first);
            n = run_of(T, W, first + steps - 1) - w0 + 1;
        }
    }
    if (lane == 0) {
        s_w0[warp] = w0;
        s_n[warp] = n;
    }
    after_the_kernel_before();                         // the parts (lengths are older: the attention waited for them)
    Join<DV> join;
    int local;
    // (one run had it all: written; none: zeros; many parts: the whole block's)
    const int many = rpb == 1 ? 8 : 32;
    if (n >= 0 && n != 1 && n <= many) {
        const size_t at = place(r, local);
        join.parts(a.ws, w0, n, local, 0, 1, lane);
        join.store(a, at, lane);
    }
    __syncthreads();
    for (int i = 0; i < rpb; ++i) {
        if (s_n[i] <= many) continue;
        const size_t at = place(r0 + i, local);
        join.parts(a.ws, s_w0[i], s_n[i], local, warp, JW, lane);
#pragma unroll
        for (int c = 0; c < join.C; ++c)
#pragma unroll
            for (int e = 0; e < join.V; ++e) s_x[warp][join.column(c, e, lane)] = join.x[c * join.V + e];
        if (lane == 0) {
            s_m[warp] = join.M;
            s_l[warp] = join.L;
        }
        __syncthreads();
        if (warp == 0) {
            float top = -INFINITY, sum = 0.f;
#pragma unroll
            for (int k = 0; k < JW; ++k) top = fmaxf(top, s_m[k]);
            const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
            for (int e = 0; e < join.C * join.V; ++e) join.x[e] = 0.f;
#pragma unroll
            for (int k = 0; k < JW; ++k) {
                const float wt = exp2_approx((s_m[k] - base) * kLog2e);
                sum = fmaf(s_l[k], wt, sum);
#pragma unroll
                for (int c = 0; c < join.C; ++c)
#pragma unroll
                    for (int e = 0; e < join.V; ++e)
                        join.x[c * join.V + e] = fmaf(s_x[k][join.column(c, e, lane)], wt, join.x[c * join.V + e]);
            }
            join.L = sum;
            join.store(a, at, lane);
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------ host

template <int DV, int JW>
cudaError_t launch_join(const Attn &a, int U, cudaStream_t stream) {
    // few rows: a block each, so that long rows are shared out; many: a warp each
    const int n_rows = a.n_seqs * a.c.Hkv * a.R;
    const int rpb = (int)(n_rows >= 2 * kGrid * JW ? JW : (n_rows + 2 * kGrid - 1) / (2 * kGrid));
    // Its blocks start as the attention kernel's end (no earlier trigger: blocks that
    // only wait would gather on the first SM that has room, and stay there).  2 x 16/4
    // x (100003, 50001) x 128: 52 us triggered at the kernel's start, 42 at its end, 44
    // as a plain launch.
    return launch_early(join_kernel<DV, JW>, dim3(((unsigned)n_rows + rpb - 1) / rpb), JW * 32, 0, stream, a, U, rpb,
                        n_rows);
}

template <int DK, int DV, bool QLO, int PM>
cudaError_t launch(const Attn &a, cudaStream_t stream) {
    using G = Geo<DK, DV>;
    static PerDeviceOnce attrs;
    cudaError_t e = attrs.run([] {
        return cudaFuncSetAttribute(attn_kernel<DK, DV, QLO, PM>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    G::SMEM);
    });
    if (e != cudaSuccess) return e;
    const int grid = a.alone ? a.n_seqs * a.c.Hkv * a.n_rb : kGrid;
    e = launch_early(attn_kernel<DK, DV, QLO, PM>, dim3(grid), G::WARPS * 32, G::SMEM, stream, a);
    if (e != cudaSuccess || a.alone) return e;
    const bool many = a.W >= 128ll * a.n_seqs * a.c.Hkv * a.n_rb;
    return many ? launch_join<DV, 16>(a, G::U, stream) : launch_join<DV, 8>(a, G::U, stream);
}

// fp32 queries keep 22 bits and give fp32 outputs or 16-bit ones alike; 16-bit
// queries are exact in one f16, and their 16-bit outputs take 11 bits of the weights.
template <int DK, int DV>
cudaError_t launch_d(const Attn &a, cudaStream_t stream) {
    if (a.q_type == GDN_DTYPE_F32) return launch<DK, DV, true, kHiLo>(a, stream);
    if (a.out_type != GDN_DTYPE_F32) return launch<DK, DV, false, kHi>(a, stream);
    return a.R <= 4 ? launch<DK, DV, false, kColumns>(a, stream) : launch<DK, DV, false, kHiLo>(a, stream);
}

template <int DK>
cudaError_t launch_k(const Attn &a, cudaStream_t stream) {
    switch (a.c.dv) {
        case 64: return launch_d<DK, 64>(a, stream);
        case 128: return launch_d<DK, 128>(a, stream);
        default: return launch_d<DK, 256>(a, stream);
    }
}

// How a call is shared out.  False where the page tables have room for 2^31 tiles
// (over all kv heads and row blocks): tiles are counted in 32 bits.
struct Plan {
    int W;                             // runs at most
    bool alone;
    size_t bytes;                      // of workspace
};
bool plan(int n_seqs, int H, int Hkv, int n_q, int dk, int dv, long long tiles, Plan *p) {
    const long long R = (long long)(H / Hkv) * n_q;
    const int warps = warps_of(dk, dv);
    const long long n_rb = (R + kRows - 1) / kRows;
    unsigned long long units, all;
    if (!host::mul_ok((unsigned long long)n_seqs, (unsigned long long)(Hkv * n_rb), &units) ||
        !host::mul_ok(units, (unsigned long long)tiles, &all) || all > (unsigned long long)INT_MAX)
        return false;
    // The lengths are on the device, so the tables' room decides.
    // Up to a unit an SM, of few tiles: a CTA each, whose warps meet in shared memory.  It
    // takes as long as 4 tiles a warp do, times how many of those the unit has; the more
    // units, the later runs over the whole GPU and a join are faster.  n tokens a sequence
    // at 128 + 128, us so and joined: 1 unit, 700: 8.5 and 9.7, 1000: 11.3 and 9.5; 32
    // units, 1000: 11.5 and 10.2; 64 units, 2200: 14.2 and 15.7, 3000: 16.9 and 16.3; 128
    // units, 4500: 22.9 and 25.2; 256 units, 16: 12.6 and 9.9.
    const long long rounds = units < 40 ? 1 : (long long)units / 20;
    p->alone = units <= (unsigned long long)kGrid && tiles <= 4 * rounds * warps;
    p->W = (int)(all < (unsigned long long)(kGrid * warps) ? all : (unsigned long long)(kGrid * warps));
    p->bytes = p->alone ? 0 : (size_t)p->W * 2 * (size_t)kRows * (dv + 2) * sizeof(float);
    return true;
}

bool sizes_ok(int n_seqs, int H, int Hkv, int n_q) {
    return n_seqs >= 0 && H >= 0 && Hkv >= 0 && n_q >= 0 && (H == 0 || (Hkv >= 1 && H % Hkv == 0));
}

}  // namespace
}  // namespace kv4
}  // namespace gdn

extern "C" {

size_t gdn_flash_attn_kv4_workspace_bytes(int n_seqs, int n_heads, int n_heads_kv, int n_q, int head_dim_k,
                                          int head_dim_v, int page_size, int max_pages) {
    using namespace gdn::kv4;
    Plan p;
    if (!sizes_ok(n_seqs, n_heads, n_heads_kv, n_q) || n_seqs == 0 || n_heads == 0 || max_pages <= 0 ||
        page_size < kTile || page_size % kTile != 0 || !gdn_flash_attn_supports(n_q, head_dim_k, head_dim_v) ||
        (long long)max_pages * page_size > INT_MAX - 64 ||
        !plan(n_seqs, n_heads, n_heads_kv, n_q, head_dim_k, head_dim_v,
              (long long)max_pages * (page_size / kTile), &p))
        return 0;
    return p.bytes;
}

int gdn_flash_attn_kv4(const void *q, const void *cache, const int *page_table, const int *seq_lens,
                       const void *mask, void *out, int n_seqs, int n_heads, int n_heads_kv, int n_q,
                       int head_dim_k, int head_dim_v, int n_pages, int page_size, int max_pages,
                       float scale, int causal, int dtype, int out_dtype, void *workspace,
                       size_t workspace_bytes, gdn_stream_t stream) {
    using namespace gdn::host;
    using namespace gdn::kv4;
    if (!sizes_ok(n_seqs, n_heads, n_heads_kv, n_q)) return GDN_ERR_ARG;
    if (dtype != GDN_DTYPE_F32 && dtype != GDN_DTYPE_BF16 && dtype != GDN_DTYPE_F16) return GDN_ERR_ARG;
    if (out_dtype != GDN_DTYPE_F32 && out_dtype != GDN_DTYPE_BF16 && out_dtype != GDN_DTYPE_F16)
        return GDN_ERR_ARG;
    if (causal != 0 && causal != 1) return GDN_ERR_ARG;
    if (!std::isfinite(scale)) return GDN_ERR_ARG;
    gdn::kv4::Span span;
    int rc = check_cache(cache, page_table, seq_lens, n_seqs, n_heads_kv, head_dim_k, head_dim_v, n_pages,
                         page_size, max_pages, &span);
    if (rc != GDN_OK) return rc;
    if (n_q > 0 && !gdn_flash_attn_supports(n_q, head_dim_k, head_dim_v)) return GDN_ERR_SHAPE;
    if (n_seqs == 0 || n_heads == 0 || n_q == 0) return GDN_OK;
    const long long cap = (long long)max_pages * page_size;
    unsigned long long rows, q_bytes, out_bytes, mask_n, mask_bytes, x;
    const unsigned long long elt = dtype == GDN_DTYPE_F32 ? 4 : 2;
    if (!mul_ok((unsigned long long)n_seqs * (unsigned long long)n_heads, (unsigned long long)n_q, &rows) ||
        rows > (unsigned long long)INT_MAX ||      // one block a row joins the parts
        !mul_ok(rows, (unsigned long long)head_dim_k, &x) || !span_bytes(x, elt, &q_bytes) ||
        !mul_ok(rows, (unsigned long long)head_dim_v, &x) ||
        !span_bytes(x, out_dtype == GDN_DTYPE_F32 ? 4 : 2, &out_bytes) ||
        !mul_ok((unsigned long long)n_seqs * (unsigned long long)n_q, (unsigned long long)cap, &mask_n) ||
        !span_bytes(mask_n, elt, &mask_bytes))
        return GDN_ERR_ARG;
    if (!q || !out) return GDN_ERR_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || (mask && !aligned(mask, elt))) return GDN_ERR_ALIGN;
    const Range ro = range_of(out, out_bytes), rc_ = range_of(cache, span.cache),
                rt = range_of(page_table, span.table), rl = range_of(seq_lens, span.lens),
                rq = range_of(q, q_bytes), rm = range_of(mask, mask ? mask_bytes : 0);
    for (Range in : {rc_, rt, rl, rq, rm})
        if (overlap(ro, in)) return GDN_ERR_ALIAS;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    Plan p;
    if (!plan(n_seqs, n_heads, n_heads_kv, n_q, head_dim_k, head_dim_v, cap / kTile, &p)) return GDN_ERR_ARG;
    const size_t need = p.bytes;
    if (workspace && need) {
        if (workspace_bytes < need || !aligned(workspace, 256)) return GDN_ERR_WORKSPACE;
        const Range rw = range_of(workspace, need);
        for (Range r : {ro, rc_, rt, rl, rq, rm})
            if (overlap(rw, r)) return GDN_ERR_ALIAS;
    }
    int *status = gdn::status_word();
    if (!status) return GDN_ERR_CUDA;
    void *ws = workspace;
    const bool owned = !ws && need;
    if (owned) {
        cudaMemPool_t pool = gdn::workspace_pool();
        if (!pool) return GDN_ERR_CUDA;
        if (cudaMallocFromPoolAsync(&ws, need, pool, st) != cudaSuccess) return GDN_ERR_NOMEM;
    }
    const int R = n_heads / n_heads_kv * n_q;
    const Attn a{{static_cast<uint8_t *>(const_cast<void *>(cache)), page_table, seq_lens, status, n_pages,
                  n_heads_kv, page_size / kTile, max_pages, head_dim_k, head_dim_v},
                 q, mask, out, static_cast<float *>(ws), n_seqs, n_heads, n_q, R,
                 (R + kRows - 1) / kRows, p.W, scale, dtype, out_dtype, causal != 0, p.alone};
    cudaError_t e;
    switch (head_dim_k) {
        case 64: e = launch_k<64>(a, st); break;
        case 128: e = launch_k<128>(a, st); break;
        default: e = launch_k<256>(a, st); break;
    }
    if (owned) {
        const cudaError_t f = cudaFreeAsync(ws, st);
        if (e == cudaSuccess) e = f;
    }
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
