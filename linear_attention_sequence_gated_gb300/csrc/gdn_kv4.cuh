// The 4-bit key / value cache: its tile format, shared by the kernels that
// write it, read it back and attend over it.
//
// Number format.  Sixteen neighbouring elements of a row share one scale s and
// each is kept as a 4-bit float (1 sign, 2 exponent, 1 mantissa bit: 0, 0.5, 1,
// 1.5, 2, 3, 4, 6) times s.  s has 5 exponent and 3 mantissa bits and no sign,
// with a 16-bit float's exponent bias, so its byte is bits 7 to 14 of s as a
// 16-bit float and one shift decodes a pair; no tensor-wide factor is needed
// for small or large rows.  A code times its scale has at most 6 significant
// bits and |value| in [2^-18, 61440]: exact in f16, bf16 and fp32 alike, so
// the decoded cache feeds f16 tensor-core MMAs without a rounding.
//
// Tile: 16 tokens of one kv head, 9 (dk + dv) bytes, in the order in which a
// warp's MMA fragments want it, so that every lane reads whole 16-byte words
// and a tile is one contiguous copy:
//   key codes    [parts of 128 (or 64) elements][16 tokens][part / 2 bytes],
//                elements in order, the even one in the low nibble;
//   key scales   [parts][16 tokens][part / 16];
//   value codes  [dv / 64 blocks r][8 g][4 t][4 w][4 bytes e]: byte e of word w
//                holds element 128 (r / 2) + L g + 8 (r % 2) + 2 w + e % 2 of
//                tokens 4 t + 2 (e / 2) (low nibble) and the next (high), with
//                L = min(16, dv / 8);
//   value scales [dv / 16 groups][16 tokens].
// Pages hold page_size / 16 tiles per kv head: cache[page][kv head][tile].
#pragma once

#include <cstdint>
#include <cstring>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

namespace gdn {
namespace kv4 {

constexpr int kTile = 16;              // tokens of a tile
constexpr int kMaxScale = 0xE2;        // scale byte of 10240: 6 * 10240 is still finite in f16
constexpr float kMaxValue = 61440.f;

__host__ __device__ constexpr int tile_bytes(int dk, int dv) { return 9 * (dk + dv); }

// The cache, its page table and lengths, as every kernel takes them.
struct View {
    uint8_t *data;          // (n_pages, Hkv, tpp, tile bytes)
    const int *table;       // (n_seqs, max_pages)
    const int *lens;        // (n_seqs)
    int *status;            // device status word
    int n_pages, Hkv, tpp, max_pages;
    int dk, dv;
};

__device__ __forceinline__ int capacity(const View &c) { return c.max_pages * c.tpp * kTile; }

// Tokens of sequence b: what the table has room for at most, none if negative.
__device__ __forceinline__ int length(const View &c, int b) {
    return min(max(c.lens[b], 0), capacity(c));
}

// Byte offset of tile `in_page` of (page, kv head h), or -1 for a page that the
// cache does not have.
__host__ __device__ inline long long tile_offset(int page, int n_pages, int Hkv, int h, int tpp,
                                                 int in_page, int bytes) {
    if ((unsigned)page >= (unsigned)n_pages) return -1;
    return (((long long)page * Hkv + h) * tpp + in_page) * bytes;
}

// Tile `tile` of (sequence b, kv head h), or NULL (recorded in the status
// word) where the table names a page that the cache does not have.
__device__ __forceinline__ uint8_t *tile_ptr(const View &c, int b, int h, int tile) {
    const int slot = tile / c.tpp;
    const int page = c.table[(size_t)b * c.max_pages + slot];
    const long long at = tile_offset(page, c.n_pages, c.Hkv, h, c.tpp, tile - slot * c.tpp,
                                     tile_bytes(c.dk, c.dv));
    if (at < 0) {
        *c.status = GDN_ERR_PAGE;
        return nullptr;
    }
    return c.data + at;
}

// Where the tokens of a call stand: they end the sequence, `raw` tokens long.
struct Place {
    int first;              // position of the call's token 0 (may be negative)
    int tile;               // the j-th tile that they can touch
    int t0;                 // the call's token at that tile's first place (may be negative)
    int count, len;         // tokens of the call; of the sequence, as far as the table reaches
    // token t of the call is one of its count, at a position that the sequence has
    __host__ __device__ bool present(int t) const {
        return t >= 0 && t < count && first + t >= 0 && first + t < len;
    }
    // the tile holds a position that the sequence has, and one of the call's tokens
    __host__ __device__ bool held() const {
        return tile >= 0 && (long long)tile * kTile < len && t0 < count;
    }
};
__host__ __device__ inline Place place_of(int raw, int cap, int count, int j) {
    Place p;
    p.count = count;
    p.len = raw < cap ? raw : cap;
    p.first = raw - count;
    p.tile = (p.first >> 4) + j;       // rounds down for a negative position too
    p.t0 = (int)((long long)p.tile * kTile - p.first);
    return p;
}

// Four code bytes -> four f16 pairs (low nibble in the low half).
__device__ __forceinline__ void decode4(uint32_t w, uint32_t (&r)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(w));
}
// Scale bytes 0, 1 (or 2, 3) of a word -> an f16 pair.
__device__ __forceinline__ uint32_t scales01(uint32_t w) { return __byte_perm(w, 0, 0x1404) >> 1; }
__device__ __forceinline__ uint32_t scales23(uint32_t w) { return __byte_perm(w, 0, 0x3424) >> 1; }

__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// (x.lo, x.lo) and (x.hi, x.hi)
__device__ __forceinline__ uint32_t dup_lo(uint32_t x) { return __byte_perm(x, 0, 0x1010); }
__device__ __forceinline__ uint32_t dup_hi(uint32_t x) { return __byte_perm(x, 0, 0x3232); }

__host__ __device__ inline float scale_value(int byte) {
    return __half2float(__ushort_as_half((unsigned short)(byte << 7)));
}

// The scale byte of a group whose largest magnitude is `a` (no NaN): a / 6
// rounded to nearest, ties to the even byte, at most kMaxScale.  The multiply
// and the conversion can be off beside a border, so the two borders around the
// candidate decide: six times a border (5 bits) is exact in fp32.
__host__ __device__ inline int scale_byte(float a) {
    a = fminf(a, kMaxValue);
    const int h = __half_as_ushort(__float2half_rn(a * (1.f / 6.f)));
    const int c = (h + 63 + ((h >> 7) & 1)) >> 7;
    const float up = 6.f * __half2float(__ushort_as_half((unsigned short)((c << 7) + 64)));
    const float dn = c > 0 ? 6.f * __half2float(__ushort_as_half((unsigned short)((c << 7) - 64))) : -1.f;
    const bool odd = c & 1;
    if (a > up || (a == up && odd)) return c + 1;
    if (a < dn || (a == dn && odd)) return c - 1;
    return c;
}

// The same for the largest magnitude of f16 or bf16 elements, whose sixth is a border
// or off it by 2^-13 of itself (2^-27 below 2^-14): the product with 2^-112 / 6 has a
// 16-bit float's exponent, so its bits from 20 on are the byte before rounding, and
// rounding them to multiples of 16 first makes borders exact (the product is within 2
// of them, and others are hundreds off).
__host__ __device__ inline int scale_byte16(float a) {
    const float t = fminf(a, kMaxValue) * 0x1.555556p-115f;
#ifdef __CUDA_ARCH__
    uint32_t u = __float_as_uint(t);
#else
    uint32_t u;
    memcpy(&u, &t, 4);
#endif
    u = (u + 8u) & ~15u;
    return (int)((u + 0x7ffffu + (u >> 20 & 1u)) >> 20);
}

// x / s as the conversion to 4 bits takes it, with r = 1 / s rounded (0 for s = 0).
// All that counts is on which side of the seven borders between codes it falls, or
// that it is one of them (ties go to the even code; a border times s is exact).
// 16-bit x: a quotient off a border is off by 2^-13 or more, and x r is within 2^-19
// of the quotient (at most 7 of interest; r may be 2 units off), so rounding x r to multiples of 2^-13,
// by adding and subtracting 1.5 * 2^10, leaves it on its side and borders exact.
__host__ __device__ inline float ratio16(float x, float r) { return fmaf(x, r, 1536.f) - 1536.f; }
// fp32 x: the correctly rounded quotient (the last step of P. Markstein, "Computation
// of elementary functions on the IBM RISC System/6000 processor", 1990, for a
// correctly rounded reciprocal), which is a border only where x / s is.
__host__ __device__ inline float ratio32(float x, float r, float s) {
    const float y = x * r;
    return fmaf(fmaf(-y, s, x), r, y);
}

#ifdef __CUDACC__
// Eight codes, the first in the lowest nibble: rounded to nearest even, at most 6.
__device__ __forceinline__ uint32_t encode8(float x0, float x1, float x2, float x3, float x4, float x5, float x6,
                                            float x7) {
    uint32_t w;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(w) : "f"(x0), "f"(x1), "f"(x2), "f"(x3), "f"(x4), "f"(x5), "f"(x6), "f"(x7));
    return w;
}
#endif

// The cache's kernels are launched as programmatic dependents, so that their blocks are
// set up while the kernel before them in the stream ends.  Every thread waits for that
// kernel's end before it reads or writes what a kernel before may write or read, so
// when this kernel has ended, so have those before it.  What they read from global
// memory they read with ordinary loads: the non-coherent kind (__ldg, ld.global.nc) is
// for data that nothing writes while the kernel runs, and these kernels are running when
// the kernel before writes the lengths or the rows; such loads, and the cache-hint
// intrinsics, are also free to move up across the wait.  Calls in a row, us: attention over
// 64 x 32/8 x 4096 x 128: 68.4 -> 65.0, one token at 64: 8.2 -> 5.5; in captured steps,
// 16 x 4 kv heads x 3000 x 128: 17.2 -> 16.6, a token's write and attention over 8 x 8 kv
// heads x 500 x 128: 12.0 -> 11.4.
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                         const A &...args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}
#ifdef __CUDACC__
__device__ __forceinline__ void after_the_kernel_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
#endif

// How the attention's work is shared out: all steps of all units (sequence, kv
// head, row block), one after another, cut into equal runs, one a warp.
// Run w of W over T steps (W <= T, so none is empty): T / W of them, one more in the
// first T % W runs; and the run of step x.
__host__ __device__ inline int run_begin(int T, int W, int w) {
    const int each = T / W, more = T - each * W;
    return each * w + (w < more ? w : more);
}
__host__ __device__ inline int run_of(int T, int W, int x) {
    const int each = T / W, more = T - each * W, big = (each + 1) * more;
    return x < big ? x / (each + 1) : more + (x - big) / each;
}
// A run that covers a unit in part leaves a partial result: in its slot 0 if
// the unit began in an earlier run, in its slot 1 if it begins in this one (so
// a run has at most one of each).
__host__ __device__ inline int partial_slot(int w, bool begins_here) { return 2 * w + (begins_here ? 1 : 0); }

}  // namespace kv4
}  // namespace gdn
