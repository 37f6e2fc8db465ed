// Decode attention over the 4-bit cache with many rows a kv head (several drafted
// queries, wide head groups): the products on the 5th-generation tensor cores.
//
// With more than 8 rows the warp-level kernel (gdn_kv4_attn.cu) decodes every tile
// again for each 8 of them, and decoding is what bounds it.  Here a CTA decodes a
// step of 128 tokens once, into f16 operand tiles in shared memory, for up to 32
// rows:
//     S^T  = K Q^T      M = 128 tokens, N = 32 rows, K = elements
//     O^T += V^T [P^T hi | P^T lo]   M = elements, N = 64, K = 128 tokens
// as tcgen05.mma (f16, fp32 accumulators in TMEM).  K is a K-major operand, V as it
// stands (token rows) an M-major one, P an N-major one, so nothing is transposed but
// V's pairs of tokens.  With tokens in TMEM lanes each thread has its own token's
// 32 scores, and the softmax needs no reduction at all as long as the maxima that
// are in use hold: a weight is 2^(score - maximum + 4), f16 takes up to 2^16, so a
// maximum is only moved (a reduction over the CTA, and a rescaling of O in TMEM) when
// a score passes it by 2^8.  Every row's maximum is set in its unit's first step.
//
// Warps: 0-3 softmax (one TMEM lane quarter each), 4-11 decode a tile of the step
// each, 12 issues the MMAs, 13 copies the tiles of later steps into a ring.  While
// the MMAs and the softmax of step i run, step i + 1 is decoded into the other pair
// of operand tiles.  Waits are bounded: one that runs out sets a flag that ends them
// all, and the status word.
#include <cmath>
#include <cstdint>

#include "gdn_kv4_attn.cuh"
#include "gdn_ptx.cuh"

namespace gdn {
namespace kv4 {
namespace {

constexpr int kTok = 128;              // tokens of a step: TMEM lanes
constexpr int kN = kManyRows;
constexpr int kDecodeWarps = 8, kMmaWarp = 12, kCopyWarp = 13, kThreads = 14 * 32;
constexpr float kBits = 4.f, kSlack = 8.f;   // weights are scaled by 2^4; scores may pass the maximum by 2^8

template <int DK, int DV>
struct Geo {
    static constexpr int TB = tile_bytes(DK, DV);
    static constexpr int ST = 3;                        // ring stages of 8 tiles
    // operand tiles: rows of 64 f16 (128 bytes, swizzled), one per 64 elements
    static constexpr int K_BYTES = kTok * DK * 2, V_BYTES = kTok * DV * 2;
    static constexpr int Q_BYTES = kN * DK * 2, P_BYTES = kTok * kN * 2;
    static constexpr int K0 = 0, V0 = K0 + 2 * K_BYTES, Q0 = V0 + 2 * V_BYTES, P0 = Q0 + 2 * Q_BYTES;
    static constexpr int RING = P0 + 2 * P_BYTES;
    static constexpr int BYTES = RING + ST * 8 * TB;
    static constexpr int SMEM = BYTES + 1024;           // (the base is rounded up)
    static_assert(SMEM <= 226 * 1024, "shared memory");
};
constexpr int kColS = 0, kColO = 2 * kN, kTmemCols = 128;   // two S tiles, O as hi | lo

// kind::f16 with f16 operands and an fp32 accumulator
constexpr uint32_t idesc(int N, bool a_mn, bool b_mn) {
    return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(kTok >> 4) << 24);
}

struct Shared {
    uint64_t full[4], raw_free[4];     // ring: copied, decoded
    uint64_t kv_full[2], kv_free[2];   // operand tiles: written, read by both products
    uint64_t s_full[2], s_free[2];     // scores: computed, read
    uint64_t p_full, p_free;           // weights: written, read (and O complete)
    uint64_t q_full, o_free;           // a unit's queries written; the last unit's O read
    uint64_t drained;                  // every product issued is complete
    uint32_t tmem;
    int stop;                          // a wait ran out
    unsigned good[8];                  // tiles of a step whose pages exist
    float f[kN], k[kN], z[kN], m[kN];  // of a row: score factor, the same in log2 units, offset, maximum
    float dz[kN];                      // what the last move took from z
    int qi[kN];                        // its query, or -1
    float red[4][kN];
};

__device__ __forceinline__ void bar_softmax() { ptx::named_sync(1, 128); }
// whether any of the 128 softmax threads says so
__device__ __forceinline__ bool any_softmax(bool x) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 2, 128, p;\n\t"
                 "selp.u32 %0, 1, 0, q;\n\t}" : "=r"(r) : "r"((uint32_t)x) : "memory");
    return r != 0;
}

template <int DK, int DV>
__global__ void __launch_bounds__(kThreads, 1) rows_kernel(const Attn a) {
    using G = Geo<DK, DV>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024 - (ptx::smem_u32(smem_raw) & 1023)) & 1023);
    __shared__ __align__(16) Shared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        sh.stop = 0;
        for (int i = 0; i < G::ST; ++i) {
            ptx::mbar_init(&sh.full[i], 1);
            ptx::mbar_init(&sh.raw_free[i], kDecodeWarps);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&sh.kv_full[i], kDecodeWarps);
            ptx::mbar_init(&sh.kv_free[i], 1);
            ptx::mbar_init(&sh.s_full[i], 1);
            ptx::mbar_init(&sh.s_free[i], 4);
        }
        ptx::mbar_init(&sh.p_full, 4);
        ptx::mbar_init(&sh.p_free, 1);
        ptx::mbar_init(&sh.q_full, 4);
        ptx::mbar_init(&sh.o_free, 4);
        ptx::mbar_init(&sh.drained, 1);
        ptx::fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        ptx::tmem_alloc(&sh.tmem, kTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = sh.tmem;
    // (whole warp, and one answer for it: its lanes stay together whatever happens)
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (__all_sync(0xffffffffu, ptx::mbar_wait(bar, parity & 1, &sh.stop))) return true;
        *const_cast<volatile int *>(&sh.stop) = 1;
        *a.c.status = GDN_ERR_TIMEOUT;
        return false;
    };

    const int units = a.c.Hkv * a.n_rb;
    const int T = steps_before(a, units, a.n_seqs, lane), W = min(a.W, T), w = blockIdx.x;
    const bool works = w < W;
    Cursor c;
    c.left = 0;
    if (works) c = run_of_call(a, units, T, W, w, lane);
    if (works && tid == 0 && __ldg(a.c.lens + c.b) > capacity(a.c)) *a.c.status = GDN_ERR_PAGE;

    if (warp == kCopyWarp) {
        // ------------------------------------------------------------ copies
        int i = 0;
        for (; c.left > 0; ++i, c.step(a, units, 1)) {
            const int st = i % G::ST;
            if (!wait(&sh.raw_free[st], i / G::ST + 1)) break;
            const int tile = c.j * 8 + lane, tiles = (c.len + kTile - 1) / kTile;
            const uint8_t *src = lane < 8 && tile < tiles ? tile_ptr(a.c, c.b, c.u / a.n_rb, tile) : nullptr;
            const unsigned have = __ballot_sync(0xffffffffu, src != nullptr);
            if (lane == 0) {
                sh.good[i & 7] = have;
                ptx::mbar_arrive_expect_tx(&sh.full[st], __popc(have) * G::TB);
            }
            __syncwarp();
            if (src) ptx::bulk_load(smem + G::RING + (st * 8 + lane) * G::TB, src, G::TB, &sh.full[st]);
        }
        // a wait that ran out: copies in flight still write this block's shared memory
        const int never = 0;
        if (c.left > 0)
            for (int k = max(0, i - G::ST); k < i; ++k)
                ptx::mbar_wait(&sh.full[k % G::ST], (k / G::ST) & 1, &never, 1 << 28);
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------ products
        bool ok = true, first_of_unit = false;
        int i = 0, unit = -1, unit_of_last = 0;
        const bool qlo = a.q_type == GDN_DTYPE_F32;
        auto second = [&](int p, bool first, int un) {          // O += V P of step p
            ok = ok && wait(&sh.p_full, p);
            if (first && un > 0) ok = ok && wait(&sh.o_free, un - 1);
            if (!ok) return;
            ptx::tc_fence_after();
            if (lane == 0) {
                const uint32_t v = ptx::smem_u32(smem + G::V0 + (p & 1) * G::V_BYTES);
                const uint32_t pw = ptx::smem_u32(smem + G::P0);
#pragma unroll
                for (int kk = 0; kk < kTok / 16; ++kk)
                    ptx::mma_bf16(tmem + kColO, ptx::smem_desc(v + kk * 2048, DV == 128 ? 16384 : 0, 1024),
                                  ptx::smem_desc(pw + kk * 1024, G::P_BYTES, 512, ptx::kSwizzle64),
                                  idesc(2 * kN, true, true), !(first && kk == 0));
                ptx::mma_commit(&sh.kv_free[p & 1]);
                ptx::mma_commit(&sh.p_free);
            }
            __syncwarp();
        };
        bool prev_first = false;
        for (; ok && c.left > 0; ++i, c.step(a, units, 1)) {
            first_of_unit = i == 0 || c.j == 0;
            bool second_done = false;
            if (first_of_unit) {
                // the softmax finishes the last unit, which needs its last product, before
                // it writes this one's queries
                if (i > 0) second(i - 1, prev_first, unit_of_last);
                second_done = true;
                ++unit;
                ok = ok && wait(&sh.q_full, unit);
            }
            ok = ok && wait(&sh.kv_full[i & 1], i >> 1) && wait(&sh.s_free[i & 1], (i >> 1) + 1);
            if (!ok) break;
            ptx::tc_fence_after();
            if (lane == 0) {
                const uint32_t k = ptx::smem_u32(smem + G::K0 + (i & 1) * G::K_BYTES);
                const uint32_t q = ptx::smem_u32(smem + G::Q0);
                const uint32_t d = tmem + kColS + (i & 1) * kN;
#pragma unroll
                for (int kk = 0; kk < DK / 16; ++kk) {
                    const uint64_t da = ptx::smem_desc(k + (kk >> 2) * 16384 + (kk & 3) * 32, 16, 1024);
                    const uint32_t bq = q + (kk >> 2) * (kN * 128) + (kk & 3) * 32;
                    ptx::mma_bf16(d, da, ptx::smem_desc(bq, 16, 1024), idesc(kN, false, false), kk > 0);
                    if (qlo)
                        ptx::mma_bf16(d, da, ptx::smem_desc(bq + G::Q_BYTES, 16, 1024), idesc(kN, false, false),
                                      true);
                }
                ptx::mma_commit(&sh.s_full[i & 1]);
            }
            __syncwarp();
            if (!second_done) second(i - 1, prev_first, unit_of_last);
            prev_first = first_of_unit;
            unit_of_last = unit;
        }
        if (i > 0) second(i - 1, prev_first, unit_of_last);
        // (after a wait that ran out there may be products that nothing waited for)
        if (lane == 0) ptx::mma_commit(&sh.drained);
        __syncwarp();
        const int never = 0;
        ptx::mbar_wait(&sh.drained, 0, &never, 1 << 28);
    } else if (warp >= 4) {
        // ------------------------------------------------------------ decode
        const int dw = warp - 4, g = lane >> 2, t = lane & 3;
        for (int i = 0; c.left > 0; ++i, c.step(a, units, 1)) {
            const int st = i % G::ST;
            if (!wait(&sh.full[st], i / G::ST) || !wait(&sh.kv_free[i & 1], (i >> 1) + 1)) break;
            const bool have = sh.good[i & 7] >> dw & 1;
            const uint8_t *p = smem + G::RING + (st * 8 + dw) * G::TB;
            uint8_t *ks = smem + G::K0 + (i & 1) * G::K_BYTES, *vs = smem + G::V0 + (i & 1) * G::V_BYTES;
            if (have) {
                // keys: lane (g, t) has elements 32 t .. (or 16 t ..) of tokens g and g + 8
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int row = g + 8 * h, r = dw * 16 + row;
                    uint8_t *dst = ks + r * 128;
                    if constexpr (DK == 128) {
                        // lanes of the second 64 elements take their words in another order,
                        // which keeps the 16-byte stores of 8 lanes on different banks
                        const int x = t >> 1 << 1;
                        const uint4 c4 = *reinterpret_cast<const uint4 *>(p + row * 64 + t * 16);
                        const uint32_t w[4] = {x ? c4.z : c4.x, x ? c4.w : c4.y, x ? c4.x : c4.z, x ? c4.y : c4.w};
                        uint32_t s2 = scales01(*reinterpret_cast<const uint16_t *>(p + 8 * DK + row * 8 + 2 * t));
                        if (x) s2 = __byte_perm(s2, 0, 0x1032);
                        const uint32_t sc[2] = {dup_lo(s2), dup_hi(s2)};
                        dst += (t >> 1) * 16384;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t y[4];
                            decode4(w[j], y);
                            const int chunk = (t & 1) * 4 + (j ^ x);
                            *reinterpret_cast<uint4 *>(dst + ((chunk ^ (r & 7)) << 4)) =
                                make_uint4(mul2(y[0], sc[j >> 1]), mul2(y[1], sc[j >> 1]), mul2(y[2], sc[j >> 1]),
                                           mul2(y[3], sc[j >> 1]));
                        }
                    } else {
                        const uint2 c2 = *reinterpret_cast<const uint2 *>(p + row * 32 + t * 8);
                        const uint32_t w[2] = {c2.x, c2.y}, sc = dup_lo(scales01(p[8 * DK + row * 4 + t]));
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            uint32_t y[4];
                            decode4(w[j], y);
                            *reinterpret_cast<uint4 *>(dst + (((2 * t + j) ^ (r & 7)) << 4)) =
                                make_uint4(mul2(y[0], sc), mul2(y[1], sc), mul2(y[2], sc), mul2(y[3], sc));
                        }
                    }
                }
            }
            // values: lane (g, t) has 8 elements a block of tokens 4 t .. 4 t + 3; a tile that
            // is not there is zeros (its weights are 0, and 0 times anything has to be)
            const int left = have ? c.len - (c.j * kTok + dw * 16 + 4 * t) : 0;
            const uint32_t live = left >= 4 ? 0xffffffffu : (left <= 0 ? 0u : (1u << (8 * left)) - 1u);
            const int swap = t >> 1;       // the same for these stores: tokens in pairs swapped
            const uint32_t sel0 = swap ? 0x7632u : 0x5410u, sel1 = swap ? 0x5410u : 0x7632u;
#pragma unroll
            for (int q = 0; q < DV / 64; ++q) {
                const uint8_t *v = p + 9 * DK;
                uint4 w4 = make_uint4(0, 0, 0, 0);
                uint32_t sw = 0;
                if (have) {
                    w4 = *reinterpret_cast<const uint4 *>(v + ((q * 8 + g) * 4 + t) * 16);
                    sw = *reinterpret_cast<const uint32_t *>(v + 8 * DV + (DV == 64 ? g >> 1 : g) * 16 + 4 * t) & live;
                }
                const uint32_t s01 = scales01(sw), s23 = scales23(sw), w[4] = {w4.x, w4.y, w4.z, w4.w};
                uint32_t y[4][4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t x[4];
                    decode4(w[e], x);
                    const uint32_t a0 = mul2(x[0], s01), a1 = mul2(x[1], s01), b0 = mul2(x[2], s23), b1 = mul2(x[3], s23);
                    y[0][e] = __byte_perm(a0, a1, sel0);
                    y[1][e] = __byte_perm(a0, a1, sel1);
                    y[2][e] = __byte_perm(b0, b1, sel0);
                    y[3][e] = __byte_perm(b0, b1, sel1);
                }
                const int el = DV == 64 ? 8 * g : 16 * g + 8 * q;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int r = dw * 16 + 4 * t + (k ^ swap);
                    *reinterpret_cast<uint4 *>(vs + (el >> 6) * 16384 + r * 128 + (((el >> 3 & 7) ^ (r & 7)) << 4)) =
                        make_uint4(y[k][0], y[k][1], y[k][2], y[k][3]);
                }
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                ptx::mbar_arrive(&sh.kv_full[i & 1]);
                ptx::mbar_arrive(&sh.raw_free[st]);
            }
        }
    } else {
        // ------------------------------------------------------------ softmax
        const uint32_t quarter = tmem + ((uint32_t)(warp * 32) << 16);
        bool ok = true;
        int i = 0, unit = 0;
        while (ok && c.left > 0) {
            const int b = c.b, hk = c.u / a.n_rb, rb = c.u - hk * a.n_rb, j0 = c.j, rep = a.H / a.c.Hkv;
            const int j1 = min(c.n, c.j + c.left), stop = min(c.len, j1 * kTok);
            const int raw = max(__ldg(a.c.lens + b), 0), n_rows = min(kN, a.R - rb * kN), n8 = (n_rows + 7) / 8;
            const int all = a.mask ? 0 : (a.causal ? min(c.len, max(raw - a.n_q + 1, 0)) : c.len);
            // queries: 4 threads a row, scaled to 2^14 by a power of two, f16 (and the remainder)
            {
                const int row = tid >> 2, part = tid & 3, real = rb * kN + row;
                constexpr int E = DK / 4;              // elements of a thread
                const bool f32 = a.q_type == GDN_DTYPE_F32;
                const size_t q0 = ((size_t)(b * (size_t)a.H + hk * rep) * a.n_q + (row < n_rows ? real : 0)) * DK + part * E;
                const uint4 *at = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(a.q) + q0 * (f32 ? 4 : 2));
                uint4 words[E / 4];
#pragma unroll
                for (int e = 0; e < E / 4; ++e)
                    words[e] = row < n_rows && (f32 || e < E / 8) ? __ldg(at + e) : make_uint4(0, 0, 0, 0);
                float x[E];
#pragma unroll
                for (int e = 0; e < E / 8; ++e) {
                    if (f32) {
                        const uint32_t v[8] = {words[2 * e].x, words[2 * e].y, words[2 * e].z, words[2 * e].w,
                                               words[2 * e + 1].x, words[2 * e + 1].y, words[2 * e + 1].z,
                                               words[2 * e + 1].w};
#pragma unroll
                        for (int h = 0; h < 8; ++h) x[8 * e + h] = __uint_as_float(v[h]);
                    } else {
                        const uint32_t v[4] = {words[e].x, words[e].y, words[e].z, words[e].w};
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            const float2 y = a.q_type == GDN_DTYPE_BF16
                                ? make_float2(__uint_as_float(v[h] << 16), __uint_as_float(v[h] & 0xffff0000u))
                                : __half22float2(*reinterpret_cast<const __half2 *>(&v[h]));
                            x[8 * e + 2 * h] = y.x;
                            x[8 * e + 2 * h + 1] = y.y;
                        }
                    }
                }
                float big = 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e) big = fmaxf(big, fabsf(x[e]));
                big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
                big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
                const int ex = min(max((int)(__float_as_uint(big) >> 23) - 127, -100), 126);
                const float up = __uint_as_float((uint32_t)(14 - ex + 127) << 23) * (a.scale < 0.f ? -1.f : 1.f);
                const float back = __uint_as_float((uint32_t)(ex - 14 + 127) << 23) * fabsf(a.scale);
#pragma unroll
                for (int e = 0; e < E; e += 8) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int h = 0; h < 4; ++h) split2(x[e + 2 * h] * up, x[e + 2 * h + 1] * up, hi[h], lo[h]);
                    const int el = part * E + e;
                    uint8_t *d = smem + G::Q0 + (el >> 6) * (kN * 128) + row * 128 + (((el >> 3 & 7) ^ (row & 7)) << 4);
                    *reinterpret_cast<uint4 *>(d) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4 *>(d + G::Q_BYTES) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
                if (part == 0) {
                    sh.f[row] = back;
                    sh.k[row] = back * kLog2e;
                    sh.m[row] = -INFINITY;
                    sh.z[row] = -kBits;
                    sh.qi[row] = row < n_rows ? real % a.n_q : -1;
                }
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&sh.q_full);
            }
            bar_softmax();
            float l[kN];
#pragma unroll
            for (int r = 0; r < kN; ++r) l[r] = 0.f;
            for (int j = j0; j < j1; ++j, ++i) {
                ok = wait(&sh.s_full[i & 1], i >> 1) && ok;
                ptx::tc_fence_after();
                float s[kN];
                ptx::tmem_ld16(quarter + kColS + (i & 1) * kN, *reinterpret_cast<float(*)[16]>(s));
                ptx::tmem_ld16(quarter + kColS + (i & 1) * kN + 16, *reinterpret_cast<float(*)[16]>(s + 16));
                ptx::tmem_ld_wait();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&sh.s_free[i & 1]);
                const int pos = j * kTok + tid;
                const bool plain = (j + 1) * kTok <= min(all, stop);
                const unsigned good = sh.good[i & 7];
                const bool simple = plain && good == 0xffu;
                // scores of tokens that a row does not see, and masks (in natural units, so
                // that a mask of the type's lowest value stays finite)
                if (!simple) {
                    const bool there = pos < stop && (good >> (tid >> 4) & 1);
#pragma unroll
                    for (int r = 0; r < kN; ++r) {
                        const int q = sh.qi[r];
                        const bool sees = there && q >= 0 &&
                                          (!a.causal || (long long)pos < (long long)raw - a.n_q + 1 + q);
                        float x = s[r] * sh.f[r];
                        if (!sees) x = -INFINITY;
                        else if (a.mask)
                            x += element(a.mask, a.q_type, ((size_t)b * a.n_q + q) * (size_t)capacity(a.c) + pos);
                        s[r] = x;
                    }
                }
                // Exponents of the weights under the maxima in use: without masks one FMA, in
                // place; with them differences in natural units, when they are needed.
                float top = -INFINITY;
                bool over = j == j0 || !ok;
                if (simple) {
#pragma unroll
                    for (int r = 0; r < kN; ++r)
                        if (r / 8 < n8) {
                            s[r] = fmaf(s[r], sh.k[r], -sh.z[r]);
                            top = fmaxf(top, s[r]);
                        }
                    over |= top > kBits + kSlack;
                } else {
#pragma unroll
                    for (int r = 0; r < kN; ++r)
                        if (r / 8 < n8) over |= s[r] > -INFINITY && !((s[r] - sh.m[r]) * kLog2e <= kSlack);
                }
                if (any_softmax(over)) {
                    if (any_softmax(!ok)) {            // (one answer for the four warps)
                        ok = false;
                        break;
                    }
                    // move every maximum to what it is by now
#pragma unroll
                    for (int r = 0; r < kN; ++r) {
                        if (r / 8 >= n8) continue;
                        float x = s[r];
#pragma unroll
                        for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
                        if (lane == 0) sh.red[warp][r] = x;
                    }
                    bar_softmax();
                    // this lane's row: its new maximum, and what its old weights shrink by
                    const float old = sh.m[lane], oldz = sh.z[lane];
                    float now = fmaxf(fmaxf(sh.red[0][lane], sh.red[1][lane]), fmaxf(sh.red[2][lane], sh.red[3][lane]));
                    if (simple) now = (now + oldz) * (1.f / kLog2e);
                    if (lane / 8 >= n8) now = 0.f;
                    now = fmaxf(now, old);
                    const float base = now == -INFINITY ? 0.f : now, z = __fmul_rn(base, kLog2e) - kBits;
                    const float cf = old == -INFINITY ? 0.f : exp2_approx(a.mask ? (old - base) * kLog2e : oldz - z);
                    bar_softmax();                     // all four warps have read the old ones
                    if (warp == 0) {
                        sh.m[lane] = now;
                        sh.z[lane] = z;
                        sh.dz[lane] = oldz - z;
                    }
                    bar_softmax();
#pragma unroll
                    for (int r = 0; r < kN; ++r) {
                        l[r] *= __shfl_sync(0xffffffffu, cf, r);
                        if (simple) s[r] += sh.dz[r];
                    }
                    if (j > j0) {
                        ok = wait(&sh.p_free, i - 1) && ok;    // O is complete up to here
                        ptx::tc_fence_after();
#pragma unroll
                        for (int col = 0; col < 2 * kN; col += 16) {
                            float o[16];
                            uint32_t u[16];
                            ptx::tmem_ld16(quarter + kColO + col, o);
                            ptx::tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                u[e] = __float_as_uint(o[e] * __shfl_sync(0xffffffffu, cf, (col + e) & (kN - 1)));
                            ptx::tmem_st16(quarter + kColO + col, u);
                        }
                        ptx::tmem_st_wait();
                    }
                }
                auto weight = [&](int r) {
                    if (simple) return exp2_approx(s[r]);
                    const float m = sh.m[r];
                    return exp2_approx(fmaf(s[r] - (m == -INFINITY ? 0.f : m), kLog2e, kBits));
                };
                // weights, hi and lo, as this token's row of the N-major operand
                if (i > 0) ok = wait(&sh.p_free, i - 1) && ok;
                uint8_t *prow = smem + G::P0;
#pragma unroll
                for (int r = 0; r < kN; r += 8) {
                    uint32_t hi[4] = {0, 0, 0, 0}, lo[4] = {0, 0, 0, 0};
                    if (r / 8 < n8) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float x = weight(r + 2 * e), y = weight(r + 2 * e + 1);
                            l[r + 2 * e] += x;
                            l[r + 2 * e + 1] += y;
                            split2(x, y, hi[e], lo[e]);
                        }
                    }
                    uint8_t *d = prow + ptx::sw64_offset(tid, r);
                    *reinterpret_cast<uint4 *>(d) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4 *>(d + G::P_BYTES) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
                ptx::fence_proxy_async_smem();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&sh.p_full);
            }
            if (!ok) break;                            // (decided together above)
            ok = wait(&sh.p_free, i - 1);
            ptx::tc_fence_after();
            // sums over the tokens' threads, then the unit's rows: this thread has element tid of each
            bar_softmax();                             // (the last reads of sh.red)
#pragma unroll
            for (int r = 0; r < kN; ++r) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o);
                if (lane == 0) sh.red[warp][r] = l[r];
            }
            bar_softmax();
            const bool whole = j0 == 0 && j1 == c.n;
            float *part = a.ws + (size_t)partial_slot(w, j0 == 0) * partial<DV>(kN);
#pragma unroll
            for (int col = 0; col < kN; col += 16) {
                float hi[16], lo[16];
                ptx::tmem_ld16(quarter + kColO + col, hi);
                ptx::tmem_ld16(quarter + kColO + kN + col, lo);
                ptx::tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int r = col + e, row = rb * kN + r;
                    if (r >= n_rows) continue;
                    const float sum = (sh.red[0][r] + sh.red[1][r]) + (sh.red[2][r] + sh.red[3][r]), x = hi[e] + lo[e];
                    if (whole) {
                        if (tid < DV) {
                            const size_t at = (((size_t)b * a.n_q + row % a.n_q) * a.H + hk * rep + row / a.n_q) * DV + tid;
                            const float y = sum == 0.f ? 0.f : x / sum;
                            if (a.out_type == GDN_DTYPE_F32) static_cast<float *>(a.out)[at] = y;
                            else if (a.out_type == GDN_DTYPE_BF16) static_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(y);
                            else static_cast<__half *>(a.out)[at] = __float2half_rn(y);
                        }
                    } else {
                        if (tid < DV) part[r * DV + tid] = x;
                        if (tid == 0) {
                            part[kN * DV + r] = sh.m[r];
                            part[kN * (DV + 1) + r] = sum;
                        }
                    }
                }
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&sh.o_free);
            ok = !any_softmax(!ok);                    // (rows' numbers are read: the next unit may set them)
            c.step(a, units, j1 - j0);
            ++unit;
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == kMmaWarp) ptx::tmem_dealloc(tmem, kTmemCols);
}

template <int DK, int DV>
cudaError_t launch(const Attn &a, cudaStream_t stream) {
    using G = Geo<DK, DV>;
    static PerDeviceOnce attrs;
    cudaError_t e = attrs.run([] {
        return cudaFuncSetAttribute(rows_kernel<DK, DV>, cudaFuncAttributeMaxDynamicSharedMemorySize, G::SMEM);
    });
    if (e != cudaSuccess) return e;
    rows_kernel<DK, DV><<<kGrid, kThreads, G::SMEM, stream>>>(a);
    e = cudaGetLastError();
    return e == cudaSuccess ? launch_join<DV>(a, stream) : e;
}

}  // namespace

bool many_rows_ok(int dk, int dv) { return dk <= 128 && dv <= 128; }

cudaError_t launch_many_rows(const Attn &a, cudaStream_t stream) {
    if (a.c.dk == 64) return a.c.dv == 64 ? launch<64, 64>(a, stream) : launch<64, 128>(a, stream);
    return a.c.dv == 64 ? launch<128, 64>(a, stream) : launch<128, 128>(a, stream);
}

}  // namespace kv4
}  // namespace gdn
