// Writing keys and values into the 4-bit cache and reading them back dense
// (gdn_kv4_write, gdn_kv4_read).  The format is in gdn_kv4.cuh.
//
// Both are streams: a write reads e bytes an element (2 or 4) and writes 9/16,
// a read the other way round, so HBM bounds them.  One warp takes one part of
// up to 128 elements of one tile (16 tokens of one kv head), keys or values:
//   * a key lane takes one scale group (16 elements) of a token: it reads and
//     writes whole 32-byte sectors of the rows, 8 code bytes and a scale byte,
//     and finds its scale without a shuffle;
//   * a value lane takes the 4 tokens x 16 (width 64: 8) elements whose codes
//     fill its own 32 (16) bytes of the tile, so the tile's nibble pairs, which
//     hold two tokens, never cross lanes.
// A tile that a write covers in part (the first and last of a run; every tile
// of a decode step) keeps its other tokens: key lanes of those tokens do not
// store, value lanes merge nibbles with what is there.  A tile belongs to one
// sequence and one warp, so no other thread writes it meanwhile.
#include <climits>
#include <cstdint>

#include "../../include/gdn.h"
#include "gdn_internal.h"
#include "gdn_kv4.cuh"

namespace gdn {
namespace kv4 {
namespace {

constexpr int kWarps = 4;              // warps of a block, each with a part of its own

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
    bool wide;                         // rows are 32-byte aligned
};

template <typename T> __device__ __forceinline__ float to_f32(T x);
template <> __device__ __forceinline__ float to_f32(float x) { return x; }
template <> __device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <> __device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }

struct Words8 {
    uint32_t w[8];
};
__device__ __forceinline__ Words8 load32(const void *p, bool wide) {
    Words8 x;
    if (wide) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(x.w[0]), "=r"(x.w[1]), "=r"(x.w[2]), "=r"(x.w[3]), "=r"(x.w[4]),
                       "=r"(x.w[5]), "=r"(x.w[6]), "=r"(x.w[7]) : "l"(p));
    } else {
        const uint4 a = reinterpret_cast<const uint4 *>(p)[0], b = reinterpret_cast<const uint4 *>(p)[1];
        x = {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
    }
    return x;
}
__device__ __forceinline__ void store32(void *p, const Words8 &x, bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(x.w[0]),
                     "r"(x.w[1]), "r"(x.w[2]), "r"(x.w[3]), "r"(x.w[4]), "r"(x.w[5]), "r"(x.w[6]),
                     "r"(x.w[7]) : "memory");
    } else {
        reinterpret_cast<uint4 *>(p)[0] = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
        reinterpret_cast<uint4 *>(p)[1] = make_uint4(x.w[4], x.w[5], x.w[6], x.w[7]);
    }
}

// N (8 or 16) consecutive elements of a row as fp32, a NaN as 0: the cache
// holds finite numbers only, so a token that a mask hides cannot spoil a row.
template <typename T, int N>
__device__ __forceinline__ void load_row(const T *p, bool wide, float (&x)[N]) {
    if constexpr (N * sizeof(T) == 16) {
        const uint4 a = *reinterpret_cast<const uint4 *>(p);
        const T *e = reinterpret_cast<const T *>(&a);
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = to_f32(e[i]);
    } else {
        constexpr int PER = 32 / (int)sizeof(T);
#pragma unroll
        for (int j = 0; j < N / PER; ++j) {
            const Words8 a = load32(p + j * PER, wide);
            const T *e = reinterpret_cast<const T *>(&a);
#pragma unroll
            for (int i = 0; i < PER; ++i) x[j * PER + i] = to_f32(e[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = x[i] == x[i] ? x[i] : 0.f;
}

template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half from_f32(float x) { return __float2half_rn(x); }

// N (8 or 16) consecutive elements of a row; every value is exact in T.
template <typename T, int N>
__device__ __forceinline__ void store_row(T *p, bool wide, const float (&x)[N]) {
    if constexpr (N * sizeof(T) == 16) {
        uint4 a;
        T *e = reinterpret_cast<T *>(&a);
#pragma unroll
        for (int i = 0; i < N; ++i) e[i] = from_f32<T>(x[i]);
        *reinterpret_cast<uint4 *>(p) = a;
    } else {
        constexpr int PER = 32 / (int)sizeof(T);
#pragma unroll
        for (int j = 0; j < N / PER; ++j) {
            Words8 a;
            T *e = reinterpret_cast<T *>(&a);
#pragma unroll
            for (int i = 0; i < PER; ++i) e[i] = from_f32<T>(x[j * PER + i]);
            store32(p + j * PER, a, wide);
        }
    }
}

template <int N>
__device__ __forceinline__ float amax(const float (&x)[N]) {
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) a = fmaxf(a, fabsf(x[i]));
    return a;
}

// What a warp works on.
struct Part : Place {
    int b, h;                          // sequence, kv head
    bool value;                        // values (else keys)
    int chunk;                         // which 128 elements
};

// Parts are numbered with the tile's parts innermost (they share a tile), then
// kv heads, then tiles.
__device__ __forceinline__ bool part_of(const Run &r, Part &p) {
    const int kc = r.c.dk > 128 ? 2 : 1, vc = r.c.dv > 128 ? 2 : 1, n = kc + vc;
    long long i = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int x = (int)(i % n);
    i /= n;
    p.value = x >= kc;
    p.chunk = p.value ? x - kc : x;
    p.h = (int)(i % r.c.Hkv);
    i /= r.c.Hkv;
    const int j = (int)(i % r.n_tiles);
    i /= r.n_tiles;
    if (i >= r.n_seqs) return false;
    p.b = (int)i;
    const int raw = max(__ldg(r.c.lens + p.b), 0), cap = capacity(r.c);
    if (raw > cap) *r.c.status = GDN_ERR_PAGE;
    const int count = r.counts ? min(max(__ldg(r.counts + p.b), 0), r.T) : r.T;
    static_cast<Place &>(p) = place_of(raw, cap, count, j);
    return true;
}

// One part of the write: W = 64 or 128 elements.
template <typename T, int W>
__device__ __forceinline__ void write_keys(const Run &r, const Part &p, uint8_t *tile, int lane) {
    constexpr int G = W / 16;          // scale groups, one a lane
    uint8_t *codes = tile + p.chunk * 16 * (W / 2), *scales = tile + 8 * r.c.dk + p.chunk * 16 * G;
    const T *k = static_cast<const T *>(r.k) + p.b * r.ks.seq + p.h * r.ks.head + p.chunk * W;
#pragma unroll
    for (int i = 0; i < G / 2; ++i) {
        const int tok = (lane + 32 * i) / G, g = lane % G;
        const int t = p.t0 + tok;
        if (!p.present(t)) continue;
        float x[16];
        load_row<T, 16>(k + t * r.ks.token + g * 16, r.wide, x);
        const int sb = scale_byte(amax(x));
        const float s = scale_value(sb);
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e)
            w[e / 4] |= encode2(ratio(x[2 * e], s), ratio(x[2 * e + 1], s)) << (8 * (e % 4));
        *reinterpret_cast<uint2 *>(codes + tok * (W / 2) + g * 8) = make_uint2(w[0], w[1]);
        scales[tok * G + g] = (uint8_t)sb;
    }
}

template <typename T, int W>
__device__ __forceinline__ void write_values(const Run &r, const Part &p, uint8_t *tile, int lane) {
    constexpr int N = W / 8;           // elements of a lane
    const int g = lane >> 2, t4 = lane & 3;
    const T *v = static_cast<const T *>(r.v) + p.b * r.vs.seq + p.h * r.vs.head + p.chunk * W + g * N;
    float x[4][N];
    int sb[4];
    uint32_t keep = 0, keep_s = 0;     // what the tile already has: nibbles of a word, scale bytes
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = p.t0 + 4 * t4 + i;
        if (p.present(t)) {
            load_row<T, N>(v + t * r.vs.token, r.wide, x[i]);
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e) x[i][e] = 0.f;
            keep |= 0x0f0fu << (4 * (i & 1) + 16 * (i >> 1));
            keep_s |= 0xffu << (8 * i);
        }
    }
    // width 64: a group of 16 spans two lanes, g and g ^ 1, which hold the same tokens
    float s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a = amax(x[i]);
        if constexpr (W == 64) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 4));
        sb[i] = scale_byte(a);
        s[i] = scale_value(sb[i]);
    }
    if (keep_s == 0xffffffffu) return;
    uint32_t w[W / 16];                // word i: elements 2i, 2i + 1 of the four tokens
#pragma unroll
    for (int i = 0; i < W / 16; ++i) {
        w[i] = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int el = 2 * i + (e & 1), k0 = 2 * (e >> 1);
            w[i] |= encode2(ratio(x[k0][el], s[k0]), ratio(x[k0 + 1][el], s[k0 + 1])) << (8 * e);
        }
    }
    uint8_t *part = tile + 9 * r.c.dk + p.chunk * 1024;
#pragma unroll
    for (int q = 0; q < W / 64; ++q) {
        uint4 *dst = reinterpret_cast<uint4 *>(part + ((q * 8 + g) * 4 + t4) * 16);
        uint4 a = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
        if (keep) {
            const uint4 o = *dst;
            a.x |= o.x & keep; a.y |= o.y & keep; a.z |= o.z & keep; a.w |= o.w & keep;
        }
        *dst = a;
    }
    if (W == 128 || !(g & 1)) {
        const int group = W == 64 ? g >> 1 : p.chunk * 8 + g;
        uint32_t *dst = reinterpret_cast<uint32_t *>(tile + 9 * r.c.dk + 8 * r.c.dv + group * 16 + 4 * t4);
        uint32_t a = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (!(keep_s >> (8 * i) & 1)) a |= (uint32_t)sb[i] << (8 * i);
        if (keep_s) a |= *dst & keep_s;
        *dst = a;
    }
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) write_kernel(const Run r) {
    Part p;
    if (!part_of(r, p)) return;
    if (!p.held()) return;
    uint8_t *tile = tile_ptr(r.c, p.b, p.h, p.tile);
    if (!tile) return;
    const int lane = threadIdx.x & 31;
    if (p.value) {
        if (r.c.dv == 64) write_values<T, 64>(r, p, tile, lane);
        else write_values<T, 128>(r, p, tile, lane);
    } else {
        if (r.c.dk == 64) write_keys<T, 64>(r, p, tile, lane);
        else write_keys<T, 128>(r, p, tile, lane);
    }
}

// One part of the read: rows of tokens that are not there are zeros.
template <typename T, int W>
__device__ __forceinline__ void read_keys(const Run &r, const Part &p, const uint8_t *tile, int lane) {
    constexpr int G = W / 16;
    const uint8_t *codes = tile + p.chunk * 16 * (W / 2), *scales = tile + 8 * r.c.dk + p.chunk * 16 * G;
    T *k = static_cast<T *>(r.k) + p.b * r.ks.seq + p.h * r.ks.head + p.chunk * W;
#pragma unroll
    for (int i = 0; i < G / 2; ++i) {
        const int tok = (lane + 32 * i) / G, g = lane % G;
        const int t = p.t0 + tok;
        if (t < 0 || t >= r.T) continue;
        float x[16];
        if (tile && p.present(t)) {
            const uint2 w = *reinterpret_cast<const uint2 *>(codes + tok * (W / 2) + g * 8);
            const float s = scale_value(scales[tok * G + g]);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint32_t h[4];
                decode4(j ? w.y : w.x, h);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[e]));
                    x[8 * j + 2 * e] = f.x * s;
                    x[8 * j + 2 * e + 1] = f.y * s;
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = 0.f;
        }
        store_row<T, 16>(k + t * r.ks.token + g * 16, r.wide, x);
    }
}

template <typename T, int W>
__device__ __forceinline__ void read_values(const Run &r, const Part &p, const uint8_t *tile, int lane) {
    constexpr int N = W / 8;
    const int g = lane >> 2, t4 = lane & 3;
    T *v = static_cast<T *>(r.v) + p.b * r.vs.seq + p.h * r.vs.head + p.chunk * W + g * N;
    float x[4][N];
    uint32_t sw = 0;
    if (tile) {
        const int group = W == 64 ? g >> 1 : p.chunk * 8 + g;
        sw = *reinterpret_cast<const uint32_t *>(tile + 9 * r.c.dk + 8 * r.c.dv + group * 16 + 4 * t4);
    }
    const uint8_t *part = tile + 9 * r.c.dk + p.chunk * 1024;
#pragma unroll
    for (int q = 0; q < W / 64; ++q) {
        uint4 a = make_uint4(0, 0, 0, 0);
        if (tile) a = *reinterpret_cast<const uint4 *>(part + ((q * 8 + g) * 4 + t4) * 16);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t h[4];
            decode4(w[i], h);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[e]));
                x[2 * (e >> 1)][8 * q + 2 * i + (e & 1)] = f.x;
                x[2 * (e >> 1) + 1][8 * q + 2 * i + (e & 1)] = f.y;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = p.t0 + 4 * t4 + i;
        if (t < 0 || t >= r.T) continue;
        const bool in = tile && p.present(t);
        const float s = in ? scale_value((sw >> (8 * i)) & 0xff) : 0.f;
#pragma unroll
        for (int e = 0; e < N; ++e) x[i][e] = in ? x[i][e] * s : 0.f;
        store_row<T, N>(v + t * r.vs.token, r.wide, x[i]);
    }
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) read_kernel(const Run r) {
    Part p;
    if (!part_of(r, p)) return;
    if (p.t0 >= r.T) return;
    const uint8_t *tile = nullptr;
    if (p.held()) tile = tile_ptr(r.c, p.b, p.h, p.tile);
    const int lane = threadIdx.x & 31;
    if (p.value) {
        if (r.c.dv == 64) read_values<T, 64>(r, p, tile, lane);
        else read_values<T, 128>(r, p, tile, lane);
    } else {
        if (r.c.dk == 64) read_keys<T, 64>(r, p, tile, lane);
        else read_keys<T, 128>(r, p, tile, lane);
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
cudaError_t launch(bool write, const Run &r, unsigned blocks, cudaStream_t stream) {
    if (write) write_kernel<T><<<blocks, kWarps * 32, 0, stream>>>(r);
    else read_kernel<T><<<blocks, kWarps * 32, 0, stream>>>(r);
    return cudaGetLastError();
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
    const long long parts = (dk > 128 ? 2 : 1) + (dv > 128 ? 2 : 1);
    unsigned long long items;
    if (!mul_ok((unsigned long long)n_seqs * (unsigned long long)Hkv,
                (unsigned long long)n_tiles * (unsigned long long)parts, &items) ||
        items > (unsigned long long)INT_MAX * kWarps)
        return GDN_ERR_ARG;
    int *status = status_word();
    if (!status) return GDN_ERR_CUDA;
    const bool wide = all % 32 == 0 && aligned(k, 32) && aligned(v, 32);
    const Run r{{cache, table, lens, status, n_pages, Hkv, page_size / kTile, max_pages, dk, dv},
                counts, k, v, ks, vs, n_seqs, T, n_tiles, wide};
    const unsigned blocks = (unsigned)((items + kWarps - 1) / kWarps);
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
