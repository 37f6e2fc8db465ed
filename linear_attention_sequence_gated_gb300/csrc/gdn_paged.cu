// Rotary positions, and rows written into the pages of a 16- or 32-bit cache
// (gdn_rotary, gdn_paged_write, gdn_rotary_write).
//
// One kernel moves rows (token, head) of up to three tensors, each either turned or
// copied, to a tensor of the same kind or to the slots of a cache.  Turning pairs (x, y) of a
// row by its token's angle, (x c - y s, y c + x s), costs 6 flops a pair against 4 or 8 bytes
// moved each way: HBM bounds long runs, latency short ones.
//
// A lane takes 32 bytes of a row, as two 16-byte pieces that hold whole pairs (piece p of each
// half, or two neighbouring ones), and a warp's lanes cover whole rows.  Rows that turn are shared out by
// tokens: a lane goes on to the same pieces of further heads, queries' and keys', whose angles are the same, so
// cosines and sines are computed once a lane, in registers, without a table in memory.  Rows that are
// copied are shared out one after another, whatever their token.
//
// The angle is exact modulo a turn: a frequency is kept as a fraction of a turn with 64
// bits, the product with the 32-bit position is taken modulo 2^64, and its upper 32 bits
// are the fraction of a turn, split into a quadrant and a rest of at most an eighth of a turn,
// which fp32 holds to 2^-28 of a turn.  So position 10^6 is as accurate as position 1.  On that rest the series of
// sine and cosine end after a few terms.
//
// Measured (GPU time of captured calls): 16384 tokens x 32/8 heads x 128, bf16, three axes: 54 us, 92 % of the rate of a copy;
// 64 tokens 3.1 us, a launch's latency and three loads one after another; 131072 tokens x 8 heads x 128 + 128 written: 155 us,
// as fast as a copy.
#include <climits>
#include <cmath>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <type_traits>

#include "../../include/gdn.h"
#include "gdn_internal.h"
#include "gdn_kv4.cuh"

namespace gdn {
namespace paged {
namespace {

constexpr int kWarps = 4;              // warps of a block, each with rows of its own

constexpr int kRows = 4;               // rows of a lane in flight

// Rows of one tensor, (n_tokens, heads, d), and where they go.
struct Rows {
    const uint8_t *src;
    uint8_t *dst;
    long long src_token, src_head;     // strides in bytes
    long long dst_token, dst_head, dst_page;   // of a cache: within its page, across heads, pages
    int heads;
    bool cache;
};
// How the rows of one width lie on a warp's lanes.
struct Lanes {
    int lanes, rows;                   // lanes of a row (32 bytes each), rows of a warp
};

struct Job {
    Rows turned[2];                    // queries and keys; of no heads where they are not turned
    Rows copied[3];                    // the others, one after another
    Lanes on, on_copied[3];
    int pieces;                        // lanes of a turned row that turn (the others copy)
    int tokens, heads, split;          // a warp that turns takes so many tokens, so many heads of each at a time, and
                                       // shares the tokens with split - 1 others
    int begin[4];                      // warps that turn, and those that copy the first, the second, the third behind them
    const int *positions;              // (n_axes, n_tokens)
    const uint4 *plan;                 // (r / 2): fraction of a turn (64 bits), axis
    const int *slots;                  // (n_tokens)
    int *status;
    int n_tokens, n_axes, page, n_slots;
    Divisor by_split, by_heads, by_page, by_rows[3];   // `split`, `heads`; tokens of a page; heads of the copied
};

// Where token t's rows go, or NULL: nowhere.
__device__ __forceinline__ uint8_t *place_of(const Job &job, const Rows &r, int t) {
    if (!r.cache) return r.dst + t * r.dst_token;
    const int slot = job.slots[t];
    if (slot >= job.n_slots) *job.status = GDN_ERR_PAGE;
    if (slot < 0 || slot >= job.n_slots) return nullptr;
    const int page = job.by_page.into(slot);
    return r.dst + page * r.dst_page + (slot - page * job.page) * r.dst_token;
}

template <typename T>
__device__ __forceinline__ void unpack(const uint4 &w, float (&x)[16 / sizeof(T)]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
            x[i] = __uint_as_float(u[i]);
        } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
}
template <typename T>
__device__ __forceinline__ uint4 pack(const float (&x)[16 / sizeof(T)]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
            u[i] = __float_as_uint(x[i]);
        } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t *>(&h);
        } else {
            const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// cos and sin of pos turns of a frequency, the sine's sign flipped for the inverse.  The Taylor polynomials of degree 9
// and 10 are off by less than x^11 / 11! = 2e-9 and x^12 / 12! = 2e-10 for |x| <= pi / 4.
__device__ __forceinline__ void angle(uint64_t turns, int pos, bool inverse, float &c, float &s) {
    const uint32_t f = (uint32_t)((turns * (uint64_t)(int64_t)pos) >> 32);   // fraction of a turn, 2^-32
    const uint32_t quadrant = (f + 0x20000000u) >> 30;
    const int rest = (int)(f - (quadrant << 30));                           // |rest| <= 2^29
    const float x = (float)rest * (0x1p-31f * 3.14159265358979f), x2 = x * x;
    const float sr = x * fmaf(x2, fmaf(x2, fmaf(x2, fmaf(x2, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6), 1.f);
    const float cr = fmaf(x2, fmaf(x2, fmaf(x2, fmaf(x2, fmaf(x2, -1.f / 3628800, 1.f / 40320), -1.f / 720), 1.f / 24),
                                   -0.5f), 1.f);
    c = quadrant & 1 ? sr : cr;
    s = quadrant & 1 ? cr : sr;
    if (quadrant == 1 || quadrant == 2) c = -c;
    if ((quadrant >= 2) != inverse) s = -s;
}

// E pairs (x[i], y[i]), or neighbours among x and among y.
template <typename T, bool NEIGHBOURS>
__device__ __forceinline__ void turn(uint4 &wa, uint4 &wb, const float (&c)[16 / sizeof(T)],
                                     const float (&s)[16 / sizeof(T)]) {
    constexpr int E = 16 / (int)sizeof(T);
    float a[E], b[E];
    unpack<T>(wa, a);
    unpack<T>(wb, b);
#pragma unroll
    for (int i = 0; i < E; ++i) {
        float &x = !NEIGHBOURS ? a[i] : i < E / 2 ? a[(2 * i) % E] : b[(2 * i) % E];
        float &y = !NEIGHBOURS ? b[i] : i < E / 2 ? a[(2 * i + 1) % E] : b[(2 * i + 1) % E];
        const float u = x, v = y;
        x = fmaf(u, c[i], -v * s[i]);
        y = fmaf(v, c[i], u * s[i]);
    }
    wa = pack<T>(a);
    wb = pack<T>(b);
}

// Up to kRows rows a warp holds at a time, one after another.
__device__ __forceinline__ void copy_rows(const Job &job, int which, int warp, int lane) {
    const Rows &r = job.copied[which];
    const Lanes on = job.on_copied[which];
    const int row = lane / on.lanes, at = 32 * (lane - row * on.lanes);
    if (row >= on.rows) return;
    const long long first = (long long)warp * kRows * on.rows + row, n = (long long)job.n_tokens * r.heads;
    uint4 x[kRows], y[kRows];
    uint8_t *dst[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
        const long long i = first + u * on.rows;
        dst[u] = nullptr;
        if (i >= n) continue;
        const int t = job.by_rows[which].into((int)i), h = (int)i - t * r.heads;
        const uint8_t *p = r.src + t * r.src_token + h * r.src_head + at;
        x[u] = *reinterpret_cast<const uint4 *>(p);
        y[u] = *reinterpret_cast<const uint4 *>(p + 16);
        dst[u] = place_of(job, r, t);
        if (dst[u]) dst[u] += h * r.dst_head + at;
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u)
        if (dst[u]) {
            *reinterpret_cast<uint4 *>(dst[u]) = x[u];
            *reinterpret_cast<uint4 *>(dst[u] + 16) = y[u];
        }
}

// KIND 0: copies only; 1: pairs are the halves of the turned part; 2: neighbours.
template <typename T, int KIND>
__global__ void __launch_bounds__(kWarps * 32, KIND == 0 ? 8 : 6) rows_kernel(const __grid_constant__ Job job, const bool inverse) {
    constexpr int E = 16 / (int)sizeof(T);             // elements of a piece
    kv4::after_the_kernel_before();
    const int lane = threadIdx.x & 31, warp = (int)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (KIND == 0 || warp >= job.begin[0]) {
        const int which = warp < job.begin[1] ? 0 : warp < job.begin[2] ? 1 : 2;
        if (warp < job.begin[3]) copy_rows(job, which, warp - job.begin[which], lane);
        return;
    }
    const int group = job.by_split.into(warp), part = warp - group * job.split;
    const int row = lane / job.on.lanes, piece = lane - row * job.on.lanes;
    const int ahead = job.by_heads.into(row), t = group * job.tokens + ahead;
    if (row >= job.on.rows || ahead >= job.tokens || t >= job.n_tokens) return;
    // the lane's two pieces of a row, in bytes
    const bool turned = piece < job.pieces;
    const int a = turned && KIND == 1 ? 16 * piece : 32 * piece;
    const int b = turned && KIND == 1 ? 16 * (piece + job.pieces) : 32 * piece + 16;
    float c[E], s[E];
    if (turned) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const uint4 f = job.plan[piece * E + i];
            const uint32_t axis = min(f.z, (uint32_t)job.n_axes - 1u);   // (whatever the plan says)
            angle((uint64_t)f.y << 32 | f.x, job.positions[(size_t)axis * job.n_tokens + t], inverse, c[i], s[i]);
        }
    }
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        const Rows &r = job.turned[which];
        const int step = job.heads * job.split;
        const uint8_t *src = r.src + t * r.src_token;
        int h = part * job.heads + row - ahead * job.heads;
        if (h >= r.heads) continue;
        uint8_t *dst = place_of(job, r, t);
        if (!dst) continue;
        for (; h < r.heads; h += kRows * step) {
            uint4 x[kRows], y[kRows];
#pragma unroll
            for (int u = 0; u < kRows; ++u)
                if (h + u * step < r.heads) {
                    const uint8_t *p = src + (h + u * step) * r.src_head;
                    x[u] = *reinterpret_cast<const uint4 *>(p + a);
                    y[u] = *reinterpret_cast<const uint4 *>(p + b);
                }
#pragma unroll
            for (int u = 0; u < kRows; ++u)
                if (h + u * step < r.heads) {
                    if (turned) turn<T, KIND == 2>(x[u], y[u], c, s);
                    uint8_t *p = dst + (h + u * step) * r.dst_head;
                    *reinterpret_cast<uint4 *>(p + a) = x[u];
                    *reinterpret_cast<uint4 *>(p + b) = y[u];
                }
        }
    }
}

}  // namespace

// ------------------------------------------------------------------ host

namespace {

using host::Range;

// A (n_tokens, heads, d) tensor, or a (n_pages, heads, page, d) cache, with its strides in elements.
struct Tensor {
    const void *p;
    long long token, head, page;
    int n_tokens, heads, n_pages, d;
};

// Checks strides, alignment and sizes, and gives the bytes from the first element to behind the last.
int span(const Tensor &t, unsigned long long elt, Range *out) {
    using namespace host;
    const long long st[3] = {t.token, t.head, t.page};
    const int n[3] = {t.n_tokens, t.heads, t.n_pages};
    unsigned long long total = (unsigned long long)t.d, x;
    *out = {0, 0};
    if (t.n_tokens == 0 || t.heads == 0 || t.n_pages == 0) return GDN_OK;
    for (int i = 0; i < 3; ++i) {
        if (st[i] < 0) return GDN_ERR_ARG;
        if (!mul_ok((unsigned long long)(n[i] - 1), (unsigned long long)st[i], &x) || x > (1ull << 59)) return GDN_ERR_ARG;
        total += x;
    }
    if (!span_bytes(total, elt, &x)) return GDN_ERR_ARG;
    if (!t.p) return GDN_ERR_ARG;
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && (unsigned long long)st[i] * elt % 16 != 0) return GDN_ERR_ALIGN;
    if (!aligned(t.p, 16)) return GDN_ERR_ALIGN;
    *out = range_of(t.p, x);
    return GDN_OK;
}

// Whether no two rows of an output share a byte: sorted by stride, each stride steps over all that the smaller ones reach.
bool rows_apart(const Tensor &t) {
    long long st[3] = {t.token, t.head, t.page};
    int n[3] = {t.n_tokens, t.heads, t.n_pages};
    for (int i = 0; i < 3; ++i)
        for (int j = 0; j + 1 < 3; ++j)
            if (st[j] > st[j + 1]) {
                const long long a = st[j];
                st[j] = st[j + 1];
                st[j + 1] = a;
                const int b = n[j];
                n[j] = n[j + 1];
                n[j + 1] = b;
            }
    long long reach = t.d;             // elements from the first to behind the last
    for (int i = 0; i < 3; ++i) {
        if (n[i] <= 1) continue;
        if (st[i] < reach) return false;
        reach += (long long)(n[i] - 1) * st[i];
    }
    return true;
}

// Elements from the first to behind the last that a token of a tensor, or a page of a cache, spans.
long long inner(const Tensor &t, bool cache) {
    return t.d + (t.heads - 1) * t.head + (cache ? (t.n_tokens - 1) * t.token : 0);
}

// Whether two tensors of ranges ra and rb share no byte: their ranges do not, or they take turns (heads of
// one projection's rows, keys and values of one buffer's pages): of one outer stride, their places within
// it do not.
bool apart(const Tensor &a, bool a_cache, Range ra, const Tensor &b, bool b_cache, Range rb, long long elt) {
    if (!host::overlap(ra, rb)) return true;
    const long long s = (a_cache ? a.page : a.token) * elt;
    if (s <= 0 || s != (b_cache ? b.page : b.token) * elt) return false;
    const long long by = static_cast<const char *>(b.p) - static_cast<const char *>(a.p);
    const long long off = ((by % s) + s) % s;
    return inner(a, a_cache) * elt <= off && off + inner(b, b_cache) * elt <= s;
}

bool same_tensor(const Tensor &a, const Tensor &b) {
    return a.p == b.p && (a.n_tokens <= 1 || a.token == b.token) && (a.heads <= 1 || a.head == b.head);
}

struct Call {
    Tensor in[3], out[3];              // q, k, v; of no heads where they are not part of the call
    bool turn[3], cache[3];
    const int *positions, *slots;
    const void *plan;
    int n_tokens, rot, n_axes, flags, page, n_slots, dtype;
};

int run(const Call &c, cudaStream_t stream) {
    using namespace host;
    if (c.dtype != GDN_DTYPE_F32 && c.dtype != GDN_DTYPE_BF16 && c.dtype != GDN_DTYPE_F16) return GDN_ERR_ARG;
    const unsigned long long elt = c.dtype == GDN_DTYPE_F32 ? 4 : 2;
    if (c.n_tokens < 0 || c.n_tokens > INT_MAX - 32) return GDN_ERR_ARG;     // (a warp's tokens may end 31 behind the last)
    bool any = false, turns = false, caches = false;
    for (int i = 0; i < 3; ++i) {
        const Tensor &t = c.in[i];
        if (t.heads < 0) return GDN_ERR_ARG;
        if (t.heads == 0) continue;
        if (t.d < 16 || t.d > 256 || t.d % 16 != 0) return GDN_ERR_HEADDIM;
        if (c.turn[i] && (c.rot < 0 || c.rot > t.d || c.rot % 16 != 0)) return GDN_ERR_HEADDIM;
        any = true;
        turns |= c.turn[i];
        caches |= c.cache[i];
    }
    if (turns && (c.n_axes < 1 || (c.flags & ~(GDN_ROTARY_NEIGHBOURS | GDN_ROTARY_INVERSE)))) return GDN_ERR_ARG;
    if (!any || c.n_tokens == 0) return GDN_OK;
    Range in[3], out[3], fixed[3] = {};
    for (int i = 0; i < 3; ++i) {
        int rc = span(c.in[i], elt, &in[i]);
        if (rc == GDN_OK) rc = span(c.out[i], elt, &out[i]);
        if (rc != GDN_OK) return rc;
        if (c.in[i].heads && !rows_apart(c.out[i])) return GDN_ERR_ALIAS;
    }
    turns &= c.rot > 0;
    if (turns) {
        unsigned long long n;
        if (!mul_ok((unsigned long long)c.n_axes, 4ull * (unsigned)c.n_tokens, &n)) return GDN_ERR_ARG;
        if (!c.positions || !c.plan) return GDN_ERR_ARG;
        if (!aligned(c.positions, 4) || !aligned(c.plan, 16)) return GDN_ERR_ALIGN;
        fixed[0] = range_of(c.positions, n);
        fixed[1] = range_of(c.plan, 8ull * (unsigned)c.rot);
    }
    if (caches) {
        if (!c.slots) return GDN_ERR_ARG;
        if (!aligned(c.slots, 4)) return GDN_ERR_ALIGN;
        fixed[2] = range_of(c.slots, 4ull * (unsigned)c.n_tokens);
    }
    for (int i = 0; i < 3; ++i)
        for (int j = 0; j < 3; ++j) {
            // a tensor may be turned in place
            const bool itself = i == j && !c.cache[i] && same_tensor(c.in[i], c.out[i]);
            if ((!itself && !apart(c.out[i], c.cache[i], out[i], c.in[j], false, in[j], (long long)elt)) ||
                overlap(out[i], fixed[j]) ||
                (j < i && !apart(c.out[i], c.cache[i], out[i], c.out[j], c.cache[j], out[j], (long long)elt)))
                return GDN_ERR_ALIAS;
        }
    Job job{};
    job.positions = c.positions;
    job.plan = static_cast<const uint4 *>(c.plan);
    job.slots = c.slots;
    job.n_tokens = c.n_tokens;
    job.n_axes = c.n_axes;
    job.pieces = (int)(c.rot * elt / 32);
    job.page = c.page;
    job.n_slots = c.n_slots;
    job.by_page = Divisor::of(c.page);
    job.status = status_word();
    if (!job.status) return GDN_ERR_CUDA;
    auto rows = [&](int i) {
        const Tensor &a = c.in[i], &b = c.out[i];
        const long long e = (long long)elt;
        return Rows{static_cast<const uint8_t *>(a.p), static_cast<uint8_t *>(const_cast<void *>(b.p)), a.token * e, a.head * e,
                    b.token * e, b.head * e, b.page * e, a.heads, c.cache[i]};
    };
    auto lanes = [&](int d) {
        const int n = (int)(d * elt / 32);
        return Lanes{n, 32 / n};
    };
    long long warps = 0;
    int heads = 0, copies = 0;
    for (int i = 0; i < 2; ++i)
        if (c.turn[i] && turns) {
            job.turned[i] = rows(i);
            heads = c.in[i].heads > heads ? c.in[i].heads : heads;
            if (c.in[i].heads) job.on = lanes(c.in[i].d);
        }
    if (heads) {
        // Few heads: rows of several tokens lie on a warp.  Many: warps share a token's, each with the angles again, while
        // tokens alone do not give each scheduler a warp.  (Never, up to that, up to sixteen times that; us, 32/8 heads x 128
        // bf16: 16 tokens 3.8, 2.7, 2.7; 64 3.8, 3.1, 3.1; 512 4.3, 4.1, 7.6; 2048 10.1, 10.1, 14.9; 64 x 64/8 x 256 fp32 10.8,
        // 3.8, 5.4.)
        job.heads = heads < job.on.rows ? heads : job.on.rows;
        job.tokens = job.on.rows / job.heads;
        // Behind a full GPU (24 warps an SM) two share a token's fp32 rows, for a shorter tail: of 16-bit ones a lane has
        // twice the angles for the same bytes.  (One and two, us: 5001 x 16/4 x 256, 64 of them turned, fp32 34.7 and 32.9, all of them
        // 34.1 and 33.6, 4000 32.9 and 28.3; 5001 x 32/8 x 128 bf16 20.7 and 21.5, 16384 54.0 and 58.3.)
        const long long groups = (c.n_tokens + job.tokens - 1) / job.tokens;
        const long long room = elt == 4 && groups > 152 * 24 ? 2 : (152 * 4 + groups - 1) / groups;
        const int passes = (heads + job.heads - 1) / job.heads, most = (int)(room < passes ? room : passes);
        // no warp without a row of its own
        job.split = (passes + (passes + most - 1) / most - 1) / ((passes + most - 1) / most);
        job.by_heads = Divisor::of(job.heads);
        job.by_split = Divisor::of(job.split);
        warps = groups * job.split;
    }
    job.begin[0] = (int)(warps < INT_MAX ? warps : INT_MAX);
    for (int i = 0; i < 3; ++i) {
        if (!c.in[i].heads || (c.turn[i] && turns)) continue;
        job.copied[copies] = rows(i);
        const Lanes on = job.on_copied[copies] = lanes(c.in[i].d);
        job.by_rows[copies] = Divisor::of(c.in[i].heads);
        const long long n = (long long)c.n_tokens * c.in[i].heads;
        if (n > INT_MAX) return GDN_ERR_ARG;
        warps += (n + kRows * on.rows - 1) / (kRows * on.rows);
        job.begin[++copies] = (int)(warps < INT_MAX ? warps : INT_MAX);
    }
    for (; copies < 3; ++copies) job.begin[copies + 1] = job.begin[copies];
    if (warps > INT_MAX - 32 * kWarps) return GDN_ERR_ARG;
    const long long blocks = (warps + kWarps - 1) / kWarps;
    const bool inverse = (c.flags & GDN_ROTARY_INVERSE) != 0;
    const int kind = !turns ? 0 : c.flags & GDN_ROTARY_NEIGHBOURS ? 2 : 1;
    cudaError_t e;
    auto go = [&](auto k0, auto k1, auto k2) {
        return kv4::launch_early(kind == 0 ? k0 : kind == 1 ? k1 : k2, dim3((unsigned)blocks), kWarps * 32, 0, stream,
                                 job, inverse);
    };
    if (kind == 0 && elt == 2)         // copies of 16-bit rows are alike
        e = go(rows_kernel<__half, 0>, rows_kernel<__half, 0>, rows_kernel<__half, 0>);
    else if (c.dtype == GDN_DTYPE_BF16)
        e = go(rows_kernel<__half, 0>, rows_kernel<__nv_bfloat16, 1>, rows_kernel<__nv_bfloat16, 2>);
    else if (c.dtype == GDN_DTYPE_F16)
        e = go(rows_kernel<__half, 0>, rows_kernel<__half, 1>, rows_kernel<__half, 2>);
    else
        e = go(rows_kernel<float, 0>, rows_kernel<float, 1>, rows_kernel<float, 2>);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

Tensor rows_of(const void *p, const long long *strides, int n_tokens, int heads, int d) {
    Tensor t{p, (long long)heads * d, d, 0, n_tokens, heads, 1, d};
    if (strides) {
        t.token = strides[0];
        t.head = strides[1];
    }
    return t;
}
// strides: pages, heads, tokens
Tensor cache_of(void *p, const long long *strides, int n_pages, int heads, int page, int d) {
    Tensor t{p, d, (long long)page * d, (long long)heads * page * d, page, heads, n_pages, d};
    if (strides) {
        t.page = strides[0];
        t.head = strides[1];
        t.token = strides[2];
    }
    return t;
}

// x modulo 1 in units of 2^-64, toward zero.
uint64_t fraction(double x) {
    x -= std::round(x);
    if (x >= 0.5) x -= 1.0;
    return (uint64_t)(int64_t)std::ldexp(x, 64);
}
// A frequency as a fraction of a turn, to 2 units of 2^-64: 1 / (2 pi) and the product are sums of two doubles
// (a position of 2^31 would make 2^-24 of a turn of one double's rounding).
uint64_t turn_of(double freq) {
    constexpr double hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;   // 1 / (2 pi)
    const double x = freq * hi;
    return fraction(x) + fraction(std::fma(freq, hi, -x) + freq * lo);
}

int cache_sizes(int n_pages, int page_size) {
    if (n_pages < 0) return GDN_ERR_ARG;
    if (page_size < 1) return GDN_ERR_SHAPE;
    return (long long)n_pages * page_size > INT_MAX ? GDN_ERR_ARG : GDN_OK;
}

}  // namespace
}  // namespace paged
}  // namespace gdn

extern "C" {

int gdn_rotary_plan(const double *freqs, const int *axes, int n, void *plan) {
    if (n < 0 || (n > 0 && (!freqs || !plan))) return GDN_ERR_ARG;
    for (int i = 0; i < n; ++i)
        if (!std::isfinite(freqs[i]) || (axes && axes[i] < 0)) return GDN_ERR_ARG;
    uint32_t *out = static_cast<uint32_t *>(plan);
    for (int i = 0; i < n; ++i) {
        const uint64_t f = gdn::paged::turn_of(freqs[i]);
        out[4 * i] = (uint32_t)f;
        out[4 * i + 1] = (uint32_t)(f >> 32);
        out[4 * i + 2] = axes ? (uint32_t)axes[i] : 0u;
        out[4 * i + 3] = 0;
    }
    return GDN_OK;
}

int gdn_rotary(const void *q, void *q_out, const void *k, void *k_out, const long long *strides, const int *positions,
               const void *plan, int n_tokens, int n_heads, int n_heads_kv, int head_dim, int rot_dim, int n_axes,
               int flags, int dtype, gdn_stream_t stream) {
    using namespace gdn::paged;
    Call c{};
    const void *in[2] = {q, k};
    void *out[2] = {q_out, k_out};
    const int heads[2] = {n_heads, n_heads_kv};
    for (int i = 0; i < 2; ++i) {
        c.in[i] = rows_of(in[i], strides ? strides + 4 * i : nullptr, n_tokens, heads[i], head_dim);
        c.out[i] = rows_of(out[i], strides ? strides + 4 * i + 2 : nullptr, n_tokens, heads[i], head_dim);
        c.turn[i] = true;
    }
    c.positions = positions;
    c.plan = plan;
    c.n_tokens = n_tokens;
    c.rot = rot_dim;
    c.n_axes = n_axes;
    c.flags = flags;
    c.page = 1;
    c.dtype = dtype;
    return run(c, reinterpret_cast<cudaStream_t>(stream));
}

int gdn_paged_write(const void *k, const void *v, const long long *strides, void *k_cache, void *v_cache,
                    const long long *cache_strides, const int *slots, int n_tokens, int n_heads_kv, int head_dim_k,
                    int head_dim_v, int n_pages, int page_size, int dtype, gdn_stream_t stream) {
    return gdn_rotary_write(nullptr, nullptr, k, v, nullptr, strides, k_cache, v_cache, cache_strides, nullptr, nullptr,
                            slots, n_tokens, 0, n_heads_kv, head_dim_k, head_dim_v, 0, 1, n_pages, page_size, 0, dtype,
                            stream);
}

int gdn_rotary_write(const void *q, void *q_out, const void *k, const void *v, const long long *q_strides,
                     const long long *kv_strides, void *k_cache, void *v_cache, const long long *cache_strides,
                     const int *positions, const void *plan, const int *slots, int n_tokens, int n_heads,
                     int n_heads_kv, int head_dim_k, int head_dim_v, int rot_dim, int n_axes, int n_pages,
                     int page_size, int flags, int dtype, gdn_stream_t stream) {
    using namespace gdn::paged;
    const int rc = cache_sizes(n_pages, page_size);
    if (rc != GDN_OK) return rc;
    if (flags & GDN_ROTARY_INVERSE) return GDN_ERR_ARG;
    Call c{};
    c.in[0] = rows_of(q, q_strides, n_tokens, n_heads, head_dim_k);
    c.out[0] = rows_of(q_out, q_strides ? q_strides + 2 : nullptr, n_tokens, n_heads, head_dim_k);
    c.in[1] = rows_of(k, kv_strides, n_tokens, n_heads_kv, head_dim_k);
    c.in[2] = rows_of(v, kv_strides ? kv_strides + 2 : nullptr, n_tokens, n_heads_kv, head_dim_v);
    c.out[1] = cache_of(k_cache, cache_strides, n_pages, n_heads_kv, page_size, head_dim_k);
    c.out[2] = cache_of(v_cache, cache_strides ? cache_strides + 3 : nullptr, n_pages, n_heads_kv, page_size,
                        head_dim_v);
    c.turn[0] = c.turn[1] = true;
    c.cache[1] = c.cache[2] = true;
    c.positions = positions;
    c.plan = plan;
    c.slots = slots;
    c.n_tokens = n_tokens;
    c.rot = rot_dim;
    c.n_axes = n_axes;
    c.flags = flags;
    c.page = page_size;
    c.n_slots = n_pages * page_size;
    c.dtype = dtype;
    return run(c, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
