// Writing keys and values into the 4-bit cache and reading them back dense
// (gdn_kv4_write, gdn_kv4_read).  The format is in gdn_kv4.cuh.
//
// Both are streams: a write reads e bytes an element (2 or 4) and writes 9/16,
// a read the other way round, so HBM bounds them.  One warp takes one part of
// one tile (16 tokens of one kv head), up to 128 elements of the tokens' keys or
// values (a write: of 8 tokens' keys):
//   * a key lane takes one scale group (16 elements) of a token: it reads and
//     writes whole 32-byte sectors of the rows, 8 code bytes and a scale byte,
//     and finds its scale without a shuffle;
//   * a value lane takes the 4 tokens x 16 (width 64: 8) elements whose codes
//     fill its own 32 (16) bytes of the tile, so the tile's nibble pairs, which
//     hold two tokens, never cross lanes.
// A tile that a write covers in part (the first and last of a run; every tile
// of a decode step) keeps its other tokens: key lanes of those tokens do not
// store, value lanes merge nibbles with what is there.  A tile belongs to one
// sequence and each of its bytes to one lane, so no other thread writes it meanwhile.
#include <climits>
#include <cstdint>
#include <type_traits>

#include "../../include/gdn.h"
#include "gdn_internal.h"
#include "gdn_kv4.cuh"

namespace gdn {
namespace kv4 {
namespace {

constexpr int kWarps = 4;              // warps of a block, each with parts of its own
constexpr int kGroup = 4;              // tiles of a warp in a call of kManyParts parts or more
constexpr long long kManyParts = 4 * 152 * 32;

struct Strides {
    long long seq, head, token;        // in elements; the row itself is contiguous
};

// One call of either kind: tokens 0 .. T-1 of each sequence stand at the
// positions that end its length.
struct Run {
    View c;
    const int *counts;                 // tokens of each sequence in this call, or NULL: T
    void *k, *v;                       // rows: read by a write, written by a read
    Strides ks, vs;
    int n_seqs, T, n_tiles;            // n_tiles: tiles that T tokens can touch
    int group;                         // tiles of a warp
    bool wide;                         // rows are 32-byte aligned
};

// N elements of a row in registers as they stand in memory: whole 32-byte words
// where the rows are 32-byte aligned.
template <typename T, int N>
struct Raw {
    static constexpr int W = N * (int)sizeof(T) / 4;
    uint32_t w[W];

    __device__ __forceinline__ void load(const T *p, bool wide) {
#pragma unroll
        for (int i = 0; i < W; i += 8) {
            const uint32_t *q = reinterpret_cast<const uint32_t *>(p) + i;
            if (W >= 8 && wide) {
                asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                             : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3]),
                               "=r"(w[(i + 4) % W]), "=r"(w[(i + 5) % W]), "=r"(w[(i + 6) % W]),
                               "=r"(w[(i + 7) % W]) : "l"(q));
            } else {
#pragma unroll
                for (int j = i; j < i + 8 && j < W; j += 4) {
                    const uint4 a = *reinterpret_cast<const uint4 *>(q + j - i);
                    w[j] = a.x; w[j + 1] = a.y; w[j + 2] = a.z; w[j + 3] = a.w;
                }
            }
        }
    }
    __device__ __forceinline__ void store(T *p, bool wide) const {
#pragma unroll
        for (int i = 0; i < W; i += 8) {
            uint32_t *q = reinterpret_cast<uint32_t *>(p) + i;
            if (W >= 8 && wide) {
                asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(q), "r"(w[i]),
                             "r"(w[i + 1]), "r"(w[i + 2]), "r"(w[i + 3]), "r"(w[(i + 4) % W]),
                             "r"(w[(i + 5) % W]), "r"(w[(i + 6) % W]), "r"(w[(i + 7) % W]) : "memory");
            } else {
#pragma unroll
                for (int j = i; j < i + 8 && j < W; j += 4)
                    *reinterpret_cast<uint4 *>(q + j - i) = make_uint4(w[j], w[j + 1], w[j + 2], w[j + 3]);
            }
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = 0;
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else if constexpr (std::is_same<T, __nv_bfloat16>::value)
            return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
        else return __half2float(__ushort_as_half((unsigned short)(i & 1 ? w[i / 2] >> 16 : w[i / 2])));
    }
    // Bits of the largest magnitude: infinity's, or above for a NaN, where there is one.
    __device__ __forceinline__ uint32_t top() const {
        if constexpr (sizeof(T) == 4) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < W; ++i) m = max(m, w[i] & 0x7fffffffu);
            return m;
        } else {
            using T2 = typename std::conditional<std::is_same<T, __nv_bfloat16>::value, __nv_bfloat162, __half2>::type;
            const T2 *x = reinterpret_cast<const T2 *>(w);
            T2 m = __habs2(x[0]);
#pragma unroll
            for (int i = 1; i < W; ++i) m = __hmax2_nan(m, __habs2(x[i]));
            const uint32_t u = *reinterpret_cast<const uint32_t *>(&m);
            return max(u & 0xffffu, u >> 16);
        }
    }
    static constexpr uint32_t INF = sizeof(T) == 4 ? 0x7f800000u
                                                   : std::is_same<T, __nv_bfloat16>::value ? 0x7f80u : 0x7c00u;
    // NaN to 0 and infinities to the largest number: the cache holds finite numbers
    // only, so that a token that a mask hides cannot spoil a row.
    __device__ __forceinline__ void finite() {
        constexpr uint32_t MAG = sizeof(T) == 4 ? 0x7fffffffu : 0x7fffu;
        constexpr int PER = 4 / (int)sizeof(T);
#pragma unroll
        for (int i = 0; i < W; ++i) {
            uint32_t x = 0;
#pragma unroll
            for (int e = 0; e < PER; ++e) {
                const uint32_t y = sizeof(T) == 4 ? w[i] : (w[i] >> (16 * e)) & 0xffffu, m = y & MAG;
                x |= (m < INF ? y : (m == INF ? y - 1 : 0u)) << (16 * e);
            }
            w[i] = x;
        }
    }
    __device__ __forceinline__ float top_value(uint32_t bits) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(bits);
        else if constexpr (std::is_same<T, __nv_bfloat16>::value) return __uint_as_float(bits << 16);
        else return __half2float(__ushort_as_half((unsigned short)bits));
    }
    // The largest magnitude, after making every element finite.
    __device__ __forceinline__ float amax() {
        uint32_t m = top();
        if (m >= INF) {
            finite();
            m = top();
        }
        return top_value(m);
    }
};

// A group's scale and what divides by it, for elements of type T.
template <typename T>
struct Scale {
    int byte;
    float s, r;
    __device__ __forceinline__ explicit Scale(float a) {
        byte = sizeof(T) == 4 ? scale_byte(a) : scale_byte16(a);
        s = scale_value(byte);
        if (sizeof(T) == 4) r = __frcp_rn(s);
        else asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
        if (byte == 0) r = 0.f;
    }
};
template <typename T>
__device__ __forceinline__ void ratios(float &x, float &y, const Scale<T> &sx, const Scale<T> &sy) {
    if constexpr (sizeof(T) == 4) {
        x = ratio32(x, sx.r, sx.s);
        y = ratio32(y, sy.r, sy.s);
    } else {
        // (the packed forms of these two instructions were slower: register pairs, spills)
        x = ratio16(x, sx.r);
        y = ratio16(y, sy.r);
    }
}

// f16 pairs of values to a row's type, exact in each
template <typename T, int N>
__device__ __forceinline__ void put(Raw<T, N> &x, int i, uint32_t pair) {   // elements i, i + 1 (i even)
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&pair));
    if constexpr (sizeof(T) == 4) {
        x.w[i] = __float_as_uint(f.x);
        x.w[i + 1] = __float_as_uint(f.y);
    } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        x.w[i / 2] = __byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x7632);
    } else {
        x.w[i / 2] = pair;
    }
}

// Parts of a tile, each of up to 128 elements: values of 16 tokens, keys of 16 (read)
// or 8 (write: more loads in flight for the registers they take).
__host__ __device__ constexpr unsigned key_parts(int dk, bool write) { return (dk > 128 ? 2 : 1) * (write ? 2 : 1); }
__host__ __device__ constexpr unsigned parts_of(int dk, int dv, bool write) {
    return key_parts(dk, write) + (dv > 128 ? 2 : 1);
}

// What a warp works on: a part of r.group tiles in a row.
struct Part : Place {
    int b, h;                          // sequence, kv head
    bool value;                        // values (else keys)
    int chunk;                         // which 128 elements
    int half;                          // of a written tile's keys: 0 or 8, the first of the tokens
    __device__ __forceinline__ void next() {
        ++tile;
        t0 += kTile;
    }
};

// blockIdx.y is the sequence (and those gridDim.y further on); the warps of the
// blocks in x are numbered with a tile's parts innermost, then kv heads, then tiles.
template <bool WRITE>
__device__ __forceinline__ bool part_of(const Run &r, int b, Part &p) {
    const unsigned kc = key_parts(r.c.dk, WRITE), n = parts_of(r.c.dk, r.c.dv, WRITE);
    const unsigned i = blockIdx.x * kWarps + (threadIdx.x >> 5);
    const unsigned unit = i / n, x = i - unit * n, j = unit / r.c.Hkv;
    p.value = x >= kc;
    p.chunk = p.value ? x - kc : WRITE ? x >> 1 : x;
    p.half = WRITE ? 8 * (x & 1) : 0;
    p.h = unit - j * r.c.Hkv;
    p.b = b;
    if (j * r.group >= (unsigned)r.n_tiles) return false;
    const int raw = max(r.c.lens[b], 0), cap = capacity(r.c);
    if (raw > cap) *r.c.status = GDN_ERR_PAGE;
    const int count = r.counts ? min(max(r.counts[b], 0), r.T) : r.T;
    static_cast<Place &>(p) = place_of(raw, cap, count, j * r.group);
    return true;
}

// One part of the write: W = 64 or 128 elements of 16 tokens.  Row loads are issued
// before the page table is looked at.
template <typename T, int W>
__device__ __forceinline__ void write_keys(const Run &r, const Part &p, int lane) {
    constexpr int G = W / 16, M = G / 4;   // groups a row (one a lane), passes over 8 tokens
    const T *k = static_cast<const T *>(r.k) + p.b * r.ks.seq + p.h * r.ks.head + p.chunk * W;
    const int g = lane % G;
    Raw<T, 16> x[M];
    bool in[M];
#pragma unroll
    for (int i = 0; i < M; ++i) {
        const int t = p.t0 + p.half + (lane + 32 * i) / G;
        in[i] = p.present(t);
        if (in[i]) x[i].load(k + t * r.ks.token + g * 16, r.wide);
    }
    uint8_t *tile = tile_ptr(r.c, p.b, p.h, p.tile);
    if (!tile) return;
    uint8_t *codes = tile + p.chunk * 16 * (W / 2), *scales = tile + 8 * r.c.dk + p.chunk * 16 * G;
#pragma unroll
    for (int i = 0; i < M; ++i) {
        if (!in[i]) continue;
        const int tok = p.half + (lane + 32 * i) / G;
        const Scale<T> s(x[i].amax());
        uint32_t w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                y[e] = x[i].get(8 * h + e);
                y[e + 1] = x[i].get(8 * h + e + 1);
                ratios(y[e], y[e + 1], s, s);
            }
            w[h] = encode8(y[0], y[1], y[2], y[3], y[4], y[5], y[6], y[7]);
        }
        *reinterpret_cast<uint2 *>(codes + tok * (W / 2) + g * 8) = make_uint2(w[0], w[1]);
        scales[tok * G + g] = (uint8_t)s.byte;
    }
}

template <typename T, int W>
__device__ __forceinline__ void write_values(const Run &r, const Part &p, int lane) {
    constexpr int N = W / 8;           // elements of a lane
    const int g = lane >> 2, t4 = lane & 3;
    const T *v = static_cast<const T *>(r.v) + p.b * r.vs.seq + p.h * r.vs.head + p.chunk * W + g * N;
    Raw<T, N> x[4];
    uint32_t keep = 0, keep_s = 0;     // what the tile already has: nibbles of a word, scale bytes
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = p.t0 + 4 * t4 + i;
        if (p.present(t)) {
            x[i].load(v + t * r.vs.token, r.wide);
        } else {
            x[i].zero();
            keep |= 0x0f0fu << (4 * (i & 1) + 16 * (i >> 1));
            keep_s |= 0xffu << (8 * i);
        }
    }
    uint8_t *tile = tile_ptr(r.c, p.b, p.h, p.tile);
    if (!tile) return;                 // (the whole warp's)
    uint4 *codes = reinterpret_cast<uint4 *>(tile + 9 * r.c.dk + p.chunk * 1024) + g * 4 + t4;
    const int group = W == 64 ? g >> 1 : p.chunk * 8 + g;
    uint32_t *scales = reinterpret_cast<uint32_t *>(tile + 9 * r.c.dk + 8 * r.c.dv + group * 16 + 4 * t4);
    const uint32_t had_s = keep ? *scales : 0;
    float a[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        a[i] = x[i].amax();
        // width 64: a group of 16 spans two lanes, g and g ^ 1, which hold the same tokens
        if constexpr (W == 64) a[i] = fmaxf(a[i], __shfl_xor_sync(0xffffffffu, a[i], 4));
    }
    if (keep_s == 0xffffffffu) return;
    const Scale<T> s[4] = {Scale<T>(a[0]), Scale<T>(a[1]), Scale<T>(a[2]), Scale<T>(a[3])};
    // (not unrolled: registers decide how many warps keep loads in flight)
#pragma unroll 1
    for (int q = 0; q < W / 64; ++q) {
        uint32_t w[4];                 // a word: elements e, e + 1 of the four tokens
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float y[4][2];
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int e = 0; e < 2; ++e) y[k][e] = x[k].get(2 * i + e);
#pragma unroll
            for (int k = 0; k < 4; k += 2)
#pragma unroll
                for (int e = 0; e < 2; ++e) ratios(y[k][e], y[k + 1][e], s[k], s[k + 1]);
            w[i] = encode8(y[0][0], y[1][0], y[0][1], y[1][1], y[2][0], y[3][0], y[2][1], y[3][1]);
        }
        if (keep) {
            const uint4 had = codes[q * 32];
            w[0] = (w[0] & ~keep) | (had.x & keep);
            w[1] = (w[1] & ~keep) | (had.y & keep);
            w[2] = (w[2] & ~keep) | (had.z & keep);
            w[3] = (w[3] & ~keep) | (had.w & keep);
        }
        codes[q * 32] = make_uint4(w[0], w[1], w[2], w[3]);
        if constexpr (W == 128) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int i = 0; i < Raw<T, N>::W / 2; ++i) x[k].w[i] = x[k].w[i + Raw<T, N>::W / 2];
        }
    }
    if (W == 128 || !(g & 1)) {
        const uint32_t b = (uint32_t)s[0].byte | (uint32_t)s[1].byte << 8 | (uint32_t)s[2].byte << 16 |
                           (uint32_t)s[3].byte << 24;
        *scales = (b & ~keep_s) | (had_s & keep_s);
    }
}

// 16-bit rows: 8 blocks an SM, 64 registers, 160 to 176 bytes a thread spilled; fp32 rows: 3
// blocks, 162 registers.  (8 x 16384 x 8 x 128: 130 to 134 us of a floor of 101, fp32 263 of 180.)
template <typename T>
__global__ void __launch_bounds__(kWarps * 32, sizeof(T) == 4 ? 3 : 8) write_kernel(const Run r) {
    after_the_kernel_before();
    const int lane = threadIdx.x & 31;
    for (int b = blockIdx.y; b < r.n_seqs; b += gridDim.y) {
        Part p;
        if (!part_of<true>(r, b, p)) continue;
#pragma unroll 1
        for (int n = 0; n < r.group; ++n, p.next()) {
            if (!p.held()) continue;
            if (p.value) {
                if (r.c.dv == 64) write_values<T, 64>(r, p, lane);
                else write_values<T, 128>(r, p, lane);
            } else {
                if (r.c.dk == 64) write_keys<T, 64>(r, p, lane);
                else write_keys<T, 128>(r, p, lane);
            }
        }
    }
}

// One part of the read: rows of tokens that are not there are zeros.
template <typename T, int W>
__device__ __forceinline__ void read_keys(const Run &r, const Part &p, const uint8_t *tile, int lane) {
    constexpr int G = W / 16, M = G / 2;
    const uint8_t *codes = tile + p.chunk * 16 * (W / 2), *scales = tile + 8 * r.c.dk + p.chunk * 16 * G;
    T *k = static_cast<T *>(r.k) + p.b * r.ks.seq + p.h * r.ks.head + p.chunk * W;
    const int g = lane % G;
    uint2 w[M];
    uint32_t s[M];
#pragma unroll
    for (int i = 0; i < M; ++i) {
        const int tok = (lane + 32 * i) / G;
        w[i] = make_uint2(0, 0);
        s[i] = 0;
        if (tile && p.present(p.t0 + tok)) {
            w[i] = *reinterpret_cast<const uint2 *>(codes + tok * (W / 2) + g * 8);
            s[i] = scales[tok * G + g];
        }
    }
#pragma unroll
    for (int i = 0; i < M; ++i) {
        const int t = p.t0 + (lane + 32 * i) / G;
        if (t < 0 || t >= r.T) continue;
        const uint32_t sc = s[i] << 7 | s[i] << 23;
        Raw<T, 16> x;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t h[4];
            decode4(j ? w[i].y : w[i].x, h);
#pragma unroll
            for (int e = 0; e < 4; ++e) put<T, 16>(x, 8 * j + 2 * e, mul2(h[e], sc));
        }
        x.store(k + t * r.ks.token + g * 16, r.wide);
    }
}

template <typename T, int W>
__device__ __forceinline__ void read_values(const Run &r, const Part &p, const uint8_t *tile, int lane) {
    constexpr int N = W / 8;
    const int g = lane >> 2, t4 = lane & 3;
    T *v = static_cast<T *>(r.v) + p.b * r.vs.seq + p.h * r.vs.head + p.chunk * W + g * N;
    const uint8_t *part = tile + 9 * r.c.dk + p.chunk * 1024;
    uint4 w4[W / 64];
    uint32_t sw = 0;
#pragma unroll
    for (int q = 0; q < W / 64; ++q) {
        w4[q] = make_uint4(0, 0, 0, 0);
        if (tile) w4[q] = *reinterpret_cast<const uint4 *>(part + ((q * 8 + g) * 4 + t4) * 16);
    }
    if (tile) {
        const int group = W == 64 ? g >> 1 : p.chunk * 8 + g;
        sw = *reinterpret_cast<const uint32_t *>(tile + 9 * r.c.dk + 8 * r.c.dv + group * 16 + 4 * t4);
        uint32_t gone = 0;             // nibbles of a word
#pragma unroll
        for (int i = 0; i < 4; ++i)    // absent tokens: zeros, whatever their bytes say
            if (!p.present(p.t0 + 4 * t4 + i)) {
                sw &= ~(0xffu << (8 * i));
                gone |= 0x0f0fu << (4 * (i & 1) + 16 * (i >> 1));
            }
        if (gone) {                    // (their signs too: -0 otherwise)
#pragma unroll
            for (int q = 0; q < W / 64; ++q) {
                w4[q].x &= ~gone;
                w4[q].y &= ~gone;
                w4[q].z &= ~gone;
                w4[q].w &= ~gone;
            }
        }
    }
    // pairs of tokens to pairs of elements
    Raw<T, N> x[4];
#pragma unroll
    for (int q = 0; q < W / 64; ++q) {
        const uint32_t w[4] = {w4[q].x, w4[q].y, w4[q].z, w4[q].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t h[4];
            decode4(w[i], h);
            const uint32_t s01 = scales01(sw), s23 = scales23(sw);
            const uint32_t a0 = mul2(h[0], s01), a1 = mul2(h[1], s01), b0 = mul2(h[2], s23), b1 = mul2(h[3], s23);
            const int e = 8 * q + 2 * i;
            put<T, N>(x[0], e, __byte_perm(a0, a1, 0x5410));
            put<T, N>(x[1], e, __byte_perm(a0, a1, 0x7632));
            put<T, N>(x[2], e, __byte_perm(b0, b1, 0x5410));
            put<T, N>(x[3], e, __byte_perm(b0, b1, 0x7632));
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = p.t0 + 4 * t4 + i;
        if (t >= 0 && t < r.T) x[i].store(v + t * r.vs.token, r.wide);
    }
}

// 64 registers; fp32 rows spill 172 bytes a thread.  (8 x 16384 x 8 x 128: 106 us of a floor of 101,
// fp32 208 of 180.)
template <typename T>
__global__ void __launch_bounds__(kWarps * 32, 8) read_kernel(const Run r) {
    after_the_kernel_before();
    const int lane = threadIdx.x & 31;
    for (int b = blockIdx.y; b < r.n_seqs; b += gridDim.y) {
        Part p;
        if (!part_of<false>(r, b, p)) continue;
#pragma unroll 1
        for (int n = 0; n < r.group && p.t0 < r.T; ++n, p.next()) {
            const uint8_t *tile = p.held() ? tile_ptr(r.c, p.b, p.h, p.tile) : nullptr;
            if (p.value) {
                if (r.c.dv == 64) read_values<T, 64>(r, p, tile, lane);
                else read_values<T, 128>(r, p, tile, lane);
            } else {
                if (r.c.dk == 64) read_keys<T, 64>(r, p, tile, lane);
                else read_keys<T, 128>(r, p, tile, lane);
            }
        }
    }
}

}  // namespace

// ------------------------------------------------------------------ host

int check_cache(const void *cache, const void *table, const void *lens, int n_seqs, int Hkv, int dk,
                int dv, int n_pages, int page_size, int max_pages, Span *span) {
    using namespace host;
    if (n_seqs < 0 || Hkv < 0 || n_pages < 0 || max_pages < 0) return GDN_ERR_ARG;
    if (!width_ok(dk) || !width_ok(dv)) return GDN_ERR_HEADDIM;
    if (page_size < kTile || page_size % kTile != 0) return GDN_ERR_SHAPE;
    // positions are 32-bit; a tile's worth of room is left for rounding up
    if ((long long)max_pages * page_size > INT_MAX - 64) return GDN_ERR_ARG;
    unsigned long long n;
    if (!mul_ok((unsigned long long)n_pages * (unsigned long long)Hkv,
                (unsigned long long)(page_size / kTile), &n) ||
        !span_bytes(n, (unsigned long long)tile_bytes(dk, dv), &span->cache) ||
        !span_bytes((unsigned long long)n_seqs * (unsigned long long)max_pages, 4, &span->table))
        return GDN_ERR_ARG;
    span->lens = 4ull * (unsigned long long)n_seqs;
    if (n_seqs == 0 || Hkv == 0) return GDN_OK;
    if (!lens || (span->table && !table) || (span->cache && !cache)) return GDN_ERR_ARG;
    if (!aligned(cache, 16) || !aligned(table, 4) || !aligned(lens, 4)) return GDN_ERR_ALIGN;
    return GDN_OK;
}

namespace {

// Bytes from the first element of a strided (n_seqs, Hkv, T, d) tensor to
// behind its last; false where a stride is negative or the size overflows.
bool strided_bytes(const Strides &s, int n_seqs, int Hkv, int T, int d, unsigned long long elt,
                   unsigned long long *out) {
    using namespace host;
    if (s.seq < 0 || s.head < 0 || s.token < 0) return false;
    unsigned long long total = (unsigned long long)d, x;
    const unsigned long long st[3] = {(unsigned long long)s.seq, (unsigned long long)s.head,
                                      (unsigned long long)s.token};
    const int n[3] = {n_seqs, Hkv, T};
    for (int i = 0; i < 3; ++i) {
        if (!mul_ok((unsigned long long)(n[i] - 1), st[i], &x) || x > (1ull << 61)) return false;
        total += x;
    }
    return total < (1ull << 61) && span_bytes(total, elt, out);
}

template <typename T>
cudaError_t launch(bool write, const Run &r, dim3 blocks, cudaStream_t stream) {
    return launch_early(write ? write_kernel<T> : read_kernel<T>, blocks, kWarps * 32, 0, stream, r);
}

int run(bool write, void *k, void *v, const long long *strides, uint8_t *cache, const int *table,
        const int *lens, const int *counts, int n_seqs, int T, int Hkv, int dk, int dv, int n_pages,
        int page_size, int max_pages, int dtype, cudaStream_t stream) {
    using namespace host;
    Span span;
    if (T < 0) return GDN_ERR_ARG;
    if (dtype != GDN_DTYPE_F32 && dtype != GDN_DTYPE_BF16 && dtype != GDN_DTYPE_F16) return GDN_ERR_ARG;
    const int rc = check_cache(cache, table, lens, n_seqs, Hkv, dk, dv, n_pages, page_size, max_pages, &span);
    if (rc != GDN_OK) return rc;
    if (n_seqs == 0 || Hkv == 0 || T == 0) return GDN_OK;
    if (T > INT_MAX - 64) return GDN_ERR_ARG;
    if (!k || !v) return GDN_ERR_ARG;
    const unsigned long long elt = dtype == GDN_DTYPE_F32 ? 4 : 2;
    Strides ks{(long long)Hkv * T * dk, (long long)T * dk, dk};
    Strides vs{(long long)Hkv * T * dv, (long long)T * dv, dv};
    if (strides) {
        ks = {strides[0], strides[1], strides[2]};
        vs = {strides[3], strides[4], strides[5]};
    }
    unsigned long long kb, vb;
    if (!strided_bytes(ks, n_seqs, Hkv, T, dk, elt, &kb) ||
        !strided_bytes(vs, n_seqs, Hkv, T, dv, elt, &vb))
        return GDN_ERR_ARG;
    if (!aligned(k, 16) || !aligned(v, 16) || (counts && !aligned(counts, 4))) return GDN_ERR_ALIGN;
    // low bits of every row's offset in bytes (a stride that no index uses has no say)
    unsigned long long all = 0;
    for (const Strides &s : {ks, vs})
        all |= ((unsigned long long)(n_seqs > 1 ? s.seq : 0) | (unsigned long long)(Hkv > 1 ? s.head : 0) |
                (unsigned long long)(T > 1 ? s.token : 0)) * elt;
    if (all % 16 != 0) return GDN_ERR_ALIGN;
    const Range rk = range_of(k, kb), rv = range_of(v, vb), rc_ = range_of(cache, span.cache),
                rt = range_of(table, span.table), rl = range_of(lens, span.lens),
                rn = range_of(counts, counts ? span.lens : 0);
    if (write) {
        for (Range in : {rk, rv, rt, rl, rn})
            if (overlap(rc_, in)) return GDN_ERR_ALIAS;
    } else {
        for (Range out : {rk, rv})
            for (Range in : {rc_, rt, rl, rn})
                if (overlap(out, in)) return GDN_ERR_ALIAS;
        if (overlap(rk, rv)) return GDN_ERR_ALIAS;
    }
    const int n_tiles = (int)(((long long)T + 2 * kTile - 2) / kTile);
    // one tile a warp while that leaves the GPU short of warps, else several in a row
    const long long each = (long long)Hkv * parts_of(dk, dv, write);
    const int group = (long long)n_seqs * n_tiles * each >= kManyParts ? kGroup : 1;
    const long long items = (n_tiles + group - 1) / group * each;  // of a sequence
    if (items > INT_MAX) return GDN_ERR_ARG;
    int *status = status_word();
    if (!status) return GDN_ERR_CUDA;
    const bool wide = all % 32 == 0 && aligned(k, 32) && aligned(v, 32);
    const Run r{{cache, table, lens, status, n_pages, Hkv, page_size / kTile, max_pages, dk, dv},
                counts, k, v, ks, vs, n_seqs, T, n_tiles, group, wide};
    const dim3 blocks((unsigned)((items + kWarps - 1) / kWarps), (unsigned)(n_seqs < 65535 ? n_seqs : 65535));
    cudaError_t e;
    if (dtype == GDN_DTYPE_BF16) e = launch<__nv_bfloat16>(write, r, blocks, stream);
    else if (dtype == GDN_DTYPE_F16) e = launch<__half>(write, r, blocks, stream);
    else e = launch<float>(write, r, blocks, stream);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace
}  // namespace kv4
}  // namespace gdn

extern "C" {

int gdn_kv4_supports(int head_dim_k, int head_dim_v) {
    return gdn::kv4::width_ok(head_dim_k) && gdn::kv4::width_ok(head_dim_v) ? 1 : 0;
}

size_t gdn_kv4_cache_bytes(int n_pages, int n_heads_kv, int page_size, int head_dim_k, int head_dim_v) {
    using namespace gdn::kv4;
    unsigned long long n, bytes;
    if (n_pages < 0 || n_heads_kv < 0 || page_size < kTile || page_size % kTile != 0 ||
        !gdn_kv4_supports(head_dim_k, head_dim_v) ||
        !gdn::host::mul_ok((unsigned long long)n_pages * (unsigned long long)n_heads_kv,
                           (unsigned long long)(page_size / kTile), &n) ||
        !gdn::host::span_bytes(n, (unsigned long long)tile_bytes(head_dim_k, head_dim_v), &bytes))
        return 0;
    return (size_t)bytes;
}

int gdn_kv4_write(const void *k, const void *v, const long long *strides, void *cache,
                  const int *page_table, const int *seq_lens, const int *new_lens, int n_seqs,
                  int n_new, int n_heads_kv, int head_dim_k, int head_dim_v, int n_pages,
                  int page_size, int max_pages, int dtype, gdn_stream_t stream) {
    return gdn::kv4::run(true, const_cast<void *>(k), const_cast<void *>(v), strides,
                         static_cast<uint8_t *>(cache), page_table, seq_lens, new_lens, n_seqs, n_new,
                         n_heads_kv, head_dim_k, head_dim_v, n_pages, page_size, max_pages, dtype,
                         reinterpret_cast<cudaStream_t>(stream));
}

int gdn_kv4_read(const void *cache, const int *page_table, const int *seq_lens, const int *read_lens,
                 void *k_out, void *v_out, int n_seqs, int n_tokens, int n_heads_kv, int head_dim_k,
                 int head_dim_v, int n_pages, int page_size, int max_pages, int dtype,
                 gdn_stream_t stream) {
    return gdn::kv4::run(false, k_out, v_out, nullptr,
                         static_cast<uint8_t *>(const_cast<void *>(cache)), page_table, seq_lens,
                         read_lens, n_seqs, n_tokens, n_heads_kv, head_dim_k, head_dim_v, n_pages,
                         page_size, max_pages, dtype, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
