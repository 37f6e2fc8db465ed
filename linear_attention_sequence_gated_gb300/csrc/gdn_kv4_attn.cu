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
// Work is shared out in tiles, not in sequences: the tiles of all (sequence, kv
// head, row block) units in a row are cut into equal runs, one a warp, so ragged
// batches and single long sequences load the GPU evenly.  A warp that has a unit
// to itself writes its output; otherwise it leaves (max, sum, output) in the
// workspace and a second kernel, launched as a programmatic dependent, joins the
// parts in a fixed order (results do not depend on timing).  It also writes the
// zero rows of empty sequences.
#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/gdn.h"
#include "gdn_internal.h"
#include "gdn_kv4.cuh"

namespace gdn {
namespace kv4 {
namespace {

constexpr int kGrid = 152;             // CTAs: one per SM of the GPU this is written for

// Rows of a unit's block (8 per MMA column tile) and warps of a CTA: 16 where
// 128 registers a thread hold the output tile, else 8.
constexpr int kMaxRows = 16;
constexpr int rows_of(long long R) { return R > 8 ? 16 : 8; }
constexpr int warps_of(int dk, int dv, int rows) { return rows == 8 && dk <= 128 && dv <= 128 ? 16 : 8; }

struct Attn {
    View c;
    const void *q, *mask;
    void *out;
    float *ws;
    int n_seqs, H, n_q, R, n_rb, W;    // R rows a kv head in n_rb blocks; W runs at most
    float scale;
    int q_type, out_type;
    bool causal;
};

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kPBits = 12.f;         // probabilities are scaled by 2^12
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
    if (type == GDN_DTYPE_F32) return __ldg(static_cast<const float *>(p) + i);
    const unsigned short u = __ldg(static_cast<const unsigned short *>(p) + i);
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

__device__ __forceinline__ int tiles_of(int len) { return (len + kTile - 1) / kTile; }

__device__ __forceinline__ long long warp_scan(long long n, int lane) {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, n, off);
        if (lane >= off) n += o;
    }
    return n;
}
// Tiles of all units of sequence b; whole-warp sums over all sequences, and
// over those before b.
__device__ __forceinline__ long long tiles_at(const Attn &a, int b, int units) {
    if (b >= a.n_seqs) return 0;
    if (__ldg(a.c.lens + b) > capacity(a.c)) *a.c.status = GDN_ERR_PAGE;
    return (long long)tiles_of(length(a.c, b)) * units;
}
__device__ __forceinline__ long long total_tiles(const Attn &a, int units, int lane) {
    long long n = 0;
    for (int b = lane; b < a.n_seqs; b += 32) n += tiles_at(a, b, units);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) n += __shfl_xor_sync(0xffffffffu, n, off);
    return n;
}
__device__ __forceinline__ long long tiles_before(const Attn &a, int units, int b, int lane) {
    long long n = 0;
    for (int i = lane; i < b; i += 32) n += tiles_at(a, i, units);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) n += __shfl_xor_sync(0xffffffffu, n, off);
    return n;
}
// The sequence that tile x lies in, and the tiles before that sequence.
__device__ __forceinline__ int find_tile(const Attn &a, int units, long long x, int lane, long long *before) {
    long long done = 0;
    for (int base = 0; base < a.n_seqs; base += 32) {
        const long long n = tiles_at(a, base + lane, units);
        const long long incl = warp_scan(n, lane) + done;
        const unsigned hit = __ballot_sync(0xffffffffu, incl > x);
        if (hit) {
            const int src = __ffs(hit) - 1;
            *before = __shfl_sync(0xffffffffu, incl - n, src);
            return base + src;
        }
        done = __shfl_sync(0xffffffffu, incl, 31);
    }
    *before = done;                    // not reached: x is below the total
    return a.n_seqs - 1;
}

// A partial result: [rows][DV] outputs, [rows] maxima, [rows] sums.
template <int DV, int ROWS> constexpr size_t kPartial = (size_t)ROWS * (DV + 2);

// One warp's share of one unit: an online softmax over tiles.
template <int DK, int DV, int NT, bool QLO>
struct Unit {
    static constexpr int CK = DK > 128 ? 2 : 1;        // key parts
    static constexpr int ST = DK >= 128 ? 8 : 4;       // MMA steps of a part
    static constexpr int VB = DV / 64;                 // value blocks, four M tiles each
    uint32_t qh[NT][CK * ST][2], ql[QLO ? NT : 1][CK * ST][2];
    float f[NT][2];                                    // row factors of the scores
    int lim[NT][2];                                    // tokens that the row sees
    size_t mrow[NT][2];                                // its mask row
    float m[NT][2], l[NT][2];
    float o[NT][VB * 4][4];

    __device__ __forceinline__ void begin(const Attn &a, int b, int hk, int rb, int lane) {
        const int g = lane >> 2, t = lane & 3;
        const int rep = a.H / a.c.Hkv;
        const int raw = max(__ldg(a.c.lens + b), 0), len = min(raw, capacity(a.c));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = rb * 8 * NT + nt * 8 + g;
            const bool ok = row < a.R;
            const size_t q0 = ((size_t)(b * (size_t)a.H + hk * rep) * a.n_q + (ok ? row : 0)) * DK;
            float x[CK * ST * 4];
            float big = 0.f;
#pragma unroll
            for (int c = 0; c < CK; ++c)
#pragma unroll
                for (int e = 0; e < ST * 4; ++e) {
                    const float v = ok ? element(a.q, a.q_type, q0 + c * 128 + t * ST * 4 + e) : 0.f;
                    x[c * ST * 4 + e] = v;
                    big = fmaxf(big, fabsf(v));
                }
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
            // 2^14 / (the power of two at or below the row's largest element)
            const int ex = min(max((int)(__float_as_uint(big) >> 23) - 127, -100), 126);
            const float up = __uint_as_float((uint32_t)(14 - ex + 127) << 23);
            const float back = __uint_as_float((uint32_t)(ex - 14 + 127) << 23) * a.scale;
#pragma unroll
            for (int s = 0; s < CK * ST; ++s)
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const float x0 = x[s * 4 + 2 * p] * up, x1 = x[s * 4 + 2 * p + 1] * up;
                    if constexpr (QLO) split2(x0, x1, qh[nt][s][p], ql[nt][s][p]);
                    else qh[nt][s][p] = half2_bits(__floats2half2_rn(x0, x1));
                }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                f[nt][r] = __shfl_sync(0xffffffffu, back, (2 * t + r) * 4);
                const int mine = rb * 8 * NT + nt * 8 + 2 * t + r, i = mine % a.n_q;
                // (a length past the table counts in full for the causal limit)
                const long long own = (long long)raw - (a.n_q - 1) + i;
                lim[nt][r] = mine >= a.R ? 0 : (a.causal ? (int)min((long long)len, own) : len);
                mrow[nt][r] = ((size_t)b * a.n_q + i) * (size_t)capacity(a.c);
                m[nt][r] = -INFINITY;
                l[nt][r] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < VB * 4; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
        }
    }

    // One tile: `p` its bytes, tokens pos .. pos + 15 of a sequence of len tokens.
    __device__ __forceinline__ void tile(const Attn &a, const uint8_t *p, int pos, int len, int lane) {
        const int g = lane >> 2, t = lane & 3;
        const int ka = 4 * (g >> 1) + (g & 1), kb = ka + 2;   // tokens of C rows g, g + 8
        float s[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
#pragma unroll
        for (int c = 0; c < CK; ++c) {
            uint32_t wa[ST / 2], wb[ST / 2];           // four steps' codes: two bytes each
            uint32_t sa, sb;                           // f16 scales of the lane's one or two groups
            if constexpr (ST == 8) {
                const uint4 x = *reinterpret_cast<const uint4 *>(p + c * 1024 + ka * 64 + t * 16);
                const uint4 y = *reinterpret_cast<const uint4 *>(p + c * 1024 + kb * 64 + t * 16);
                wa[0] = x.x; wa[1] = x.y; wa[2] = x.z; wa[3] = x.w;
                wb[0] = y.x; wb[1] = y.y; wb[2] = y.z; wb[3] = y.w;
                const uint8_t *sc = p + 8 * DK + c * 128 + 2 * t;
                sa = scales01(*reinterpret_cast<const uint16_t *>(sc + ka * 8));
                sb = scales01(*reinterpret_cast<const uint16_t *>(sc + kb * 8));
            } else {
                const uint2 x = *reinterpret_cast<const uint2 *>(p + ka * 32 + t * 8);
                const uint2 y = *reinterpret_cast<const uint2 *>(p + kb * 32 + t * 8);
                wa[0] = x.x; wa[1] = x.y;
                wb[0] = y.x; wb[1] = y.y;
                const uint8_t *sc = p + 8 * DK + t;
                sa = scales01(sc[ka * 4]);
                sb = scales01(sc[kb * 4]);
            }
#pragma unroll
            for (int h = 0; h < ST / 2; ++h) {         // a word a token: two steps
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
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma(s[nt], A, qh[nt][st][0], qh[nt][st][1]);
                        if constexpr (QLO) mma(s[nt], A, ql[nt][st][0], ql[nt][st][1]);
                    }
                }
            }
        }
        // scores in natural units, so that a mask of the type's lowest value stays finite
        uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int key = pos + (e < 2 ? ka : kb), r = e & 1;
                float x = s[nt][e] * f[nt][r];
                if (key < lim[nt][r]) {
                    if (a.mask) x += element(a.mask, a.q_type, mrow[nt][r] + key);
                } else {
                    x = -INFINITY;
                }
                s[nt][e] = x;
            }
            float pr[4];
            bool moved = false;
            float cf[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float mx = fmaxf(s[nt][r], s[nt][r + 2]);
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                const float mn = fmaxf(m[nt][r], mx);
                const float base = mn == -INFINITY ? 0.f : mn;
                cf[r] = exp2_approx((m[nt][r] - base) * kLog2e);
                moved |= mn != m[nt][r];
                m[nt][r] = mn;
                pr[r] = exp2_approx(fmaf(s[nt][r] - base, kLog2e, kPBits));
                pr[r + 2] = exp2_approx(fmaf(s[nt][r + 2] - base, kLog2e, kPBits));
            }
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int r = 0; r < 2; ++r) l[nt][r] *= cf[r];
#pragma unroll
                for (int i = 0; i < VB * 4; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[nt][i][e] *= cf[e & 1];
            }
            l[nt][0] += pr[0] + pr[2];
            l[nt][1] += pr[1] + pr[3];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                split2(pr[2 * k], pr[2 * k + 1], ph[nt][k], pl[nt][k]);
                ph[nt][k] = transpose8(ph[nt][k]);
                pl[nt][k] = transpose8(pl[nt][k]);
            }
        }
        // tokens behind the sequence's last: their scale bytes may hold anything,
        // and 0 times infinity would spoil the row
        const int left = len - pos - 4 * t;
        const uint32_t live = left >= 4 ? 0xffffffffu : (left <= 0 ? 0u : (1u << (8 * left)) - 1u);
#pragma unroll
        for (int r = 0; r < VB; ++r) {
            const uint4 w4 = *reinterpret_cast<const uint4 *>(p + 9 * DK + ((r * 8 + g) * 4 + t) * 16);
            const int group = DV == 64 ? g >> 1 : (r >> 1) * 8 + g;
            const uint32_t sw = *reinterpret_cast<const uint32_t *>(p + 9 * DK + 8 * DV + group * 16 + 4 * t) & live;
            const uint32_t s01 = scales01(sw), s23 = scales23(sw);
            const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t x[4];
                decode4(w[i], x);
                const uint32_t A[4] = {mul2(x[0], s01), mul2(x[1], s01), mul2(x[2], s23), mul2(x[3], s23)};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma(o[nt][r * 4 + i], A, ph[nt][0], ph[nt][1]);
                    mma(o[nt][r * 4 + i], A, pl[nt][0], pl[nt][1]);
                }
            }
        }
    }

    // The unit's rows: outputs where this warp saw all of its tiles, else a partial.
    __device__ __forceinline__ void end(const Attn &a, int b, int hk, int rb, bool whole, int slot, int lane) {
        const int g = lane >> 2, t = lane & 3, rep = a.H / a.c.Hkv;
        float *part = a.ws + (size_t)slot * kPartial<DV, 8 * NT>;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float sum = l[nt][r];
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
                const int local = nt * 8 + 2 * t + r, row = rb * 8 * NT + local;
                if (row >= a.R) continue;
                const float inv = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
                const size_t at = (((size_t)b * a.n_q + row % a.n_q) * a.H + hk * rep + row / a.n_q) * DV;
#pragma unroll
                for (int blk = 0; blk < VB; ++blk) {
                    const int el = 128 * (blk >> 1) + (DV == 64 ? 8 : 16) * g + 8 * (blk & 1);
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = o[nt][blk * 4 + e / 2][2 * (e & 1) + r] * inv;
                    if (whole) store8(a.out, a.out_type, at + el, x);
                    else store8(part, GDN_DTYPE_F32, (size_t)local * DV + el, x);
                }
                if (!whole && g == 0) {
                    part[8 * NT * DV + local] = m[nt][r];
                    part[8 * NT * (DV + 1) + local] = sum;
                }
            }
    }
};

template <int DK, int DV, int NT, bool QLO>
__global__ void __launch_bounds__(warps_of(DK, DV, 8 * NT) * 32, 1) attn_kernel(const Attn a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int units = a.c.Hkv * a.n_rb;
    const long long T = total_tiles(a, units, lane);
    const int W = (int)min((long long)a.W, T);
    // neighbouring runs on different SMs: few tiles spread over the GPU
    const int w = warp * gridDim.x + blockIdx.x;
    if (w >= W) return;
    long long at = run_begin(T, W, w);
    const long long stop = run_begin(T, W, w + 1);
    long long before;
    int b = find_tile(a, units, at, lane, &before);
    int len = length(a.c, b), n = tiles_of(len);
    int u = (int)((at - before) / n);
    int j = (int)((at - before) % n);
    Unit<DK, DV, NT, QLO> unit;
    while (at < stop) {
        const int j0 = j, j1 = (int)min((long long)n, j + (stop - at));
        const int hk = u / a.n_rb, rb = u - hk * a.n_rb;
        unit.begin(a, b, hk, rb, lane);
        for (; j < j1; ++j) {
            const uint8_t *p = tile_ptr(a.c, b, hk, j);
            if (p) unit.tile(a, p, j * kTile, len, lane);
        }
        unit.end(a, b, hk, rb, j0 == 0 && j1 == n, partial_slot(w, j0 == 0), lane);
        at += j1 - j0;
        j = 0;
        if (++u == units && at < stop) {               // next sequence that holds anything
            u = 0;
            do {
                len = length(a.c, ++b);
                n = tiles_of(len);
            } while (n == 0);
        }
    }
}

// Joins the partial results of one row: thread (p, x) adds up parts p, p + PL,
// ... of 4 columns with a running maximum, then the PL threads of a column join.
constexpr int kJoinThreads = 256;
template <int DV, int ROWS>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const Attn a) {
    constexpr int XL = DV / 4, PL = kJoinThreads / XL;
    __shared__ float sm[PL], sl[PL];
    __shared__ float4 so[PL][XL];
    const int lane = threadIdx.x & 31;
    long long i = blockIdx.x;
    const int row = (int)(i % a.R);
    i /= a.R;
    const int hk = (int)(i % a.c.Hkv), b = (int)(i / a.c.Hkv);
    const int rb = row / ROWS, local = row % ROWS;
    const int units = a.c.Hkv * a.n_rb, n = tiles_of(length(a.c, b));
    const long long T = total_tiles(a, units, lane);
    const int W = (int)min((long long)a.W, T);
    const int x = threadIdx.x % XL, p = threadIdx.x / XL;
    const size_t at = (((size_t)b * a.n_q + row % a.n_q) * a.H + hk * (a.H / a.c.Hkv) + row / a.n_q) * DV + 4 * x;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float M = -INFINITY, L = 0.f;
    const long long first = tiles_before(a, units, b, lane) + (long long)(hk * a.n_rb + rb) * n;
    // the attention kernel's results; every block waits, so that this grid never
    // ends before that one
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (n > 0) {
        const int w0 = run_of(T, W, first), w1 = run_of(T, W, first + n - 1);
        if (w0 == w1) return;                          // one run had it all and wrote it
        for (int w = w0 + p; w <= w1; w += PL) {
            const float *part = a.ws + (size_t)partial_slot(w, w == w0) * kPartial<DV, ROWS>;
            const float m = __ldcg(part + ROWS * DV + local), l = __ldcg(part + ROWS * (DV + 1) + local);
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(part + local * DV) + x);
            const float mn = fmaxf(M, m), base = mn == -INFINITY ? 0.f : mn;
            const float c0 = exp2_approx((M - base) * kLog2e), c1 = exp2_approx((m - base) * kLog2e);
            acc = make_float4(acc.x * c0 + v.x * c1, acc.y * c0 + v.y * c1, acc.z * c0 + v.z * c1,
                              acc.w * c0 + v.w * c1);
            L = L * c0 + l * c1;
            M = mn;
        }
    }
    so[p][x] = acc;
    if (x == 0) {
        sm[p] = M;
        sl[p] = L;
    }
    __syncthreads();
    if (p != 0) return;
    float top = -INFINITY;
#pragma unroll
    for (int i2 = 0; i2 < PL; ++i2) top = fmaxf(top, sm[i2]);
    const float base = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i2 = 0; i2 < PL; ++i2) {
        const float c = exp2_approx((sm[i2] - base) * kLog2e);
        const float4 v = so[i2][x];
        sum += sl[i2] * c;
        acc = make_float4(acc.x + v.x * c, acc.y + v.y * c, acc.z + v.z * c, acc.w + v.w * c);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    if (a.out_type == GDN_DTYPE_F32) {
        *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at) = acc;
    } else if (a.out_type == GDN_DTYPE_BF16) {
        __nv_bfloat162 h[2] = {__floats2bfloat162_rn(acc.x, acc.y), __floats2bfloat162_rn(acc.z, acc.w)};
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + at) = *reinterpret_cast<uint2 *>(h);
    } else {
        __half2 h[2] = {__floats2half2_rn(acc.x, acc.y), __floats2half2_rn(acc.z, acc.w)};
        *reinterpret_cast<uint2 *>(static_cast<__half *>(a.out) + at) = *reinterpret_cast<uint2 *>(h);
    }
}

// ------------------------------------------------------------------ host

template <int DK, int DV, int NT, bool QLO>
cudaError_t launch(const Attn &a, cudaStream_t stream) {
    const int warps = warps_of(DK, DV, 8 * NT);
    attn_kernel<DK, DV, NT, QLO><<<kGrid, warps * 32, 0, stream>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)a.n_seqs * a.c.Hkv * a.R));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, join_kernel<DV, 8 * NT>, a);
}

template <int DK, int DV>
cudaError_t launch_d(const Attn &a, cudaStream_t stream) {
    const bool lo = a.q_type == GDN_DTYPE_F32;
    if (rows_of(a.R) == 8) return lo ? launch<DK, DV, 1, true>(a, stream) : launch<DK, DV, 1, false>(a, stream);
    return lo ? launch<DK, DV, 2, true>(a, stream) : launch<DK, DV, 2, false>(a, stream);
}

template <int DK>
cudaError_t launch_k(const Attn &a, cudaStream_t stream) {
    switch (a.c.dv) {
        case 64: return launch_d<DK, 64>(a, stream);
        case 128: return launch_d<DK, 128>(a, stream);
        default: return launch_d<DK, 256>(a, stream);
    }
}

// Runs and workspace of a call; false where the tile count passes what the
// schedule's 64-bit products hold.
bool plan(int n_seqs, int H, int Hkv, int n_q, int dk, int dv, long long tiles, int *W, size_t *bytes) {
    const long long R = (long long)(H / Hkv) * n_q;
    const int rows = rows_of(R);
    const long long n_rb = (R + rows - 1) / rows;
    unsigned long long units, all;
    if (!host::mul_ok((unsigned long long)n_seqs, (unsigned long long)(Hkv * n_rb), &units) ||
        !host::mul_ok(units, (unsigned long long)tiles, &all) || all > (1ull << 48))
        return false;
    const int most = kGrid * warps_of(dk, dv, rows);
    *W = (int)(all < (unsigned long long)most ? all : (unsigned long long)most);
    *bytes = (size_t)*W * 2 * (size_t)rows * (dv + 2) * sizeof(float);
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
    int W;
    size_t bytes;
    if (!sizes_ok(n_seqs, n_heads, n_heads_kv, n_q) || n_seqs == 0 || n_heads == 0 || max_pages <= 0 ||
        page_size < kTile || page_size % kTile != 0 || !gdn_flash_attn_supports(n_q, head_dim_k, head_dim_v) ||
        (long long)max_pages * page_size > INT_MAX - 64 ||
        !plan(n_seqs, n_heads, n_heads_kv, n_q, head_dim_k, head_dim_v,
              (long long)max_pages * (page_size / kTile), &W, &bytes))
        return 0;
    return bytes;
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
    if (cap == 0)                                      // no room for a token: every row is zero
        return cudaMemsetAsync(out, 0, out_bytes, st) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
    int W;
    size_t need;
    if (!plan(n_seqs, n_heads, n_heads_kv, n_q, head_dim_k, head_dim_v, cap / kTile, &W, &need))
        return GDN_ERR_ARG;
    if (workspace) {
        if (workspace_bytes < need || !aligned(workspace, 256)) return GDN_ERR_WORKSPACE;
        const Range rw = range_of(workspace, need);
        for (Range r : {ro, rc_, rt, rl, rq, rm})
            if (overlap(rw, r)) return GDN_ERR_ALIAS;
    }
    int *status = gdn::status_word();
    if (!status) return GDN_ERR_CUDA;
    void *ws = workspace;
    if (!ws) {
        cudaMemPool_t pool = gdn::workspace_pool();
        if (!pool) return GDN_ERR_CUDA;
        if (cudaMallocFromPoolAsync(&ws, need, pool, st) != cudaSuccess) return GDN_ERR_NOMEM;
    }
    const int R = n_heads / n_heads_kv * n_q;
    const Attn a{{static_cast<uint8_t *>(const_cast<void *>(cache)), page_table, seq_lens, status, n_pages,
                  n_heads_kv, page_size / kTile, max_pages, head_dim_k, head_dim_v},
                 q, mask, out, static_cast<float *>(ws), n_seqs, n_heads, n_q, R,
                 (R + rows_of(R) - 1) / rows_of(R), W, scale, dtype, out_dtype, causal != 0};
    cudaError_t e;
    switch (head_dim_k) {
        case 64: e = launch_k<64>(a, st); break;
        case 128: e = launch_k<128>(a, st); break;
        default: e = launch_k<256>(a, st); break;
    }
    if (!workspace) {
        const cudaError_t f = cudaFreeAsync(ws, st);
        if (e == cudaSuccess) e = f;
    }
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
