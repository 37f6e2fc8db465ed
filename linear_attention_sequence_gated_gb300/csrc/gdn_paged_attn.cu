// gdn_flash_attn_paged: checks, tensor maps and the choice between clusters and runs (the kernels are in
// gdn_paged_attn.cuh).
#include <climits>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "../../include/gdn.h"
#include "gdn_internal.h"
#include "gdn_paged_attn.cuh"

namespace gdn {
namespace paged {
namespace {

constexpr int kMaxQueries = 19;

typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                             const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static EncodeFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess && q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeFn>(p);
    });
    return fn;
}

// A cache (n_pages, heads, page, d) as a tensor map takes it: the three outer dimensions by ascending
// strides, each of which has to hold a whole number of the one below it.
struct Layout {
    unsigned long long dim[3], stride[3];   // strides in bytes
    int order;                              // two bits a dimension: 0 token, 1 head, 2 page
    unsigned long long bytes;               // from the first element to behind the last
};

int layout_of(const long long *strides, int n_pages, int heads, int page, int d, unsigned long long elt, Layout *out) {
    const unsigned long long n[3] = {(unsigned long long)page, (unsigned long long)heads, (unsigned long long)n_pages};
    unsigned long long st[3] = {};
    if ((long long)heads * page > 1ll << 36) return GDN_ERR_ARG;
    const long long dense[3] = {d, (long long)page * d, (long long)heads * page * d};
    for (int i = 0; i < 3; ++i) {
        const long long x = strides ? strides[2 - i] : dense[i];      // given as page, head, token
        if (x < 0 || x > 1ll << 40) {
            if (n[i] > 1) return GDN_ERR_ARG;
            continue;
        }
        st[i] = (unsigned long long)x * elt;
    }
    int at[3] = {0, 1, 2};
    // a dimension of one element has no stride to speak of: outermost
    auto key = [&](int i) { return n[i] > 1 ? st[i] : ~0ull; };
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2; ++j)
            if (key(at[j]) > key(at[j + 1])) {
                const int x = at[j];
                at[j] = at[j + 1];
                at[j + 1] = x;
            }
    unsigned long long below = (unsigned long long)d * elt, reach = below, unit = 16;
    out->order = 0;
    for (int i = 0; i < 3; ++i) {
        const int a = at[i];
        const unsigned long long s = n[a] > 1 ? st[a] : (below + unit - 1) / unit * unit;
        if (s % 16 != 0) return GDN_ERR_ALIGN;
        if (s < below || (i > 0 && s % unit != 0)) return GDN_ERR_SHAPE;
        if (s >= 1ull << 40) return GDN_ERR_ARG;
        out->dim[i] = n[a];
        out->stride[i] = s;
        out->order |= a << (2 * i);
        reach += (n[a] - 1) * s;
        below = n[a] * s;
        unit = s;
        if (below > 1ull << 56) return GDN_ERR_ARG;
    }
    out->bytes = reach;
    return GDN_OK;
}

bool make_map(CUtensorMap *map, const void *p, const Layout &x, int d, int dtype) {
    EncodeFn enc = encode_fn();
    if (!enc) return false;
    const cuuint32_t wide = dtype == GDN_DTYPE_F32 ? 32 : 64;
    cuuint64_t dims[4] = {(cuuint64_t)d}, strides[3];
    cuuint32_t box[4] = {wide, 1, 1, 1};
    const cuuint32_t each[4] = {1, 1, 1, 1};
    for (int i = 0; i < 3; ++i) {
        dims[i + 1] = x.dim[i];
        strides[i] = x.stride[i];
        if ((x.order >> (2 * i) & 3) == 0) box[i + 1] = kTile;
    }
    const CUtensorMapDataType type = dtype == GDN_DTYPE_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                     : dtype == GDN_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                               : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    return enc(map, type, 4, const_cast<void *>(p), dims, strides, box, each, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How a call is shared out.
struct Plan {
    Share share;
    int cluster, grid;
    size_t bytes;                      // of the workspace
};

// CTAs a unit, or 0 for equal runs, by the room that the tables have (the lengths are on the device): what the
// slowest CTA streams, in bytes, and as bytes the time of what does not overlap it: each wave of CTAs' start and
// join, 4 us; a cluster's join, 2 us; for runs 11 us once, the second kernel's among them.  Each group of a
// cluster's CTAs has a tile at least.  One CTA fits on an SM, and fewer clusters fit on the GPU's partitions than
// SMs allow for (16 clusters of 8 x 250 tiles of 16 KB are two waves: 29 us, in runs 19).  Runs adapt to lengths below the
// tables' room, so clusters have to be ahead by an eighth.  (Runs and clusters, us, 32/8 heads x 128: 1 x 1000 tokens 9.0 and 8.0, 1 x 4000 10.8 and 10.2,
// 1 x 16000 19.7 and 21.1, 1 x 60000 45 and 60; 16 x 1000 20.9 and 14.5, 38 x 1500 47 and 43.)
constexpr int kAtOnce[4] = {kGrid, 76, 36, 15};        // clusters of 1, 2, 4 and 8 CTAs
static_assert(kMaxCluster == 8, "sizes");
constexpr long long kWaveCost = 160 << 10, kClusterCost = 80 << 10, kRunsCost = 448 << 10;
bool plan_of(int n_seqs, int H, int Hkv, int n_q, int dk, int dv, int page, int max_pages, int elt, Plan *p) {
    p->share = share_of(dk, dv, elt, H / Hkv * n_q);
    const long long units = (long long)n_seqs * Hkv * p->share.units, groups = p->share.groups;
    const long long tiles = ((long long)max_pages * page + kTile - 1) / kTile;
    const long long steps = tiles ? tiles + kUnitCost : 0;
    // (steps are rounded up to whole groups)
    if (units > INT_MAX || steps > INT_MAX || (steps > 0 && units > (INT_MAX - 16) / steps)) return false;
    const long long stage = (long long)kTile * (dk + dv) * elt;
    long long cl = 1, by_cluster = 0;
    for (int i = 0; i < 4; ++i) {
        const long long c = 1ll << i, waves = (units + kAtOnce[i] - 1) / kAtOnce[i];
        const long long cost = waves * ((tiles + c - 1) / c * stage + kWaveCost + (i ? kClusterCost : 0));
        if (i && (tiles <= c * groups || cost >= by_cluster)) continue;
        by_cluster = cost;
        cl = c;
    }
    const long long by_runs = (units * steps + kGrid - 1) / kGrid * stage + kRunsCost;
    p->cluster = by_cluster + by_cluster / 8 <= by_runs ? (int)cl : 0;
    const long long runs = (units * steps + groups - 1) / groups;
    p->grid = p->cluster ? (int)(units * cl) : (int)(runs < kGrid ? runs : kGrid);
    p->bytes = p->cluster || p->grid < 2 ? 0
                                         : p->grid * (2 * partial_size(p->share.blocks * kBlock, dv) * sizeof(float) +
                                                      sizeof(int) * 4);
    return units * cl <= INT_MAX;
}

bool width_ok(int d) { return d == 64 || d == 128 || d == 256; }

}  // namespace
}  // namespace paged
}  // namespace gdn

extern "C" {

int gdn_flash_attn_paged_supports(int n_q, int head_dim_k, int head_dim_v) {
    using namespace gdn::paged;
    return n_q >= 1 && n_q <= kMaxQueries && width_ok(head_dim_k) && width_ok(head_dim_v) ? 1 : 0;
}

size_t gdn_flash_attn_paged_workspace_bytes(int n_seqs, int n_heads, int n_heads_kv, int n_q, int head_dim_k,
                                            int head_dim_v, int page_size, int max_pages, int dtype) {
    using namespace gdn::paged;
    Plan p;
    if (n_seqs < 1 || n_heads < 1 || n_heads_kv < 1 || n_heads % n_heads_kv != 0 || max_pages < 1 ||
        !gdn_flash_attn_paged_supports(n_q, head_dim_k, head_dim_v) || page_size < kTile || page_size % kTile != 0 ||
        (long long)max_pages * page_size > INT_MAX - 64 || dtype < GDN_DTYPE_F32 || dtype > GDN_DTYPE_F16 ||
        (long long)(n_heads / n_heads_kv) * n_q > INT_MAX - 64 ||
        !plan_of(n_seqs, n_heads, n_heads_kv, n_q, head_dim_k, head_dim_v, page_size, max_pages,
                 dtype == GDN_DTYPE_F32 ? 4 : 2, &p))
        return 0;
    return p.bytes;
}

int gdn_flash_attn_paged(const void *q, const long long *q_strides, const void *k_cache, const void *v_cache,
                         const long long *cache_strides, const int *page_table, const int *seq_lens, const void *mask,
                         void *out, int n_seqs, int n_heads, int n_heads_kv, int n_q, int head_dim_k, int head_dim_v,
                         int n_pages, int page_size, int max_pages, float scale, int causal, int dtype, int out_dtype,
                         void *workspace, size_t workspace_bytes, gdn_stream_t stream) {
    using namespace gdn::host;
    using namespace gdn::paged;
    using gdn::Divisor;
    if (n_seqs < 0 || n_heads < 0 || n_heads_kv < 0 || n_q < 0 || n_pages < 0 || max_pages < 0) return GDN_ERR_ARG;
    if (dtype != GDN_DTYPE_F32 && dtype != GDN_DTYPE_BF16 && dtype != GDN_DTYPE_F16) return GDN_ERR_ARG;
    if (out_dtype != GDN_DTYPE_F32 && out_dtype != GDN_DTYPE_BF16 && out_dtype != GDN_DTYPE_F16) return GDN_ERR_ARG;
    if (causal != 0 && causal != 1) return GDN_ERR_ARG;
    if (!std::isfinite(scale)) return GDN_ERR_ARG;
    if (n_heads > 0 && (n_heads_kv < 1 || n_heads % n_heads_kv != 0)) return GDN_ERR_ARG;
    if (!width_ok(head_dim_k) || !width_ok(head_dim_v)) return GDN_ERR_HEADDIM;
    if (n_q > kMaxQueries || page_size < kTile || page_size % kTile != 0) return GDN_ERR_SHAPE;
    if ((long long)max_pages * page_size > INT_MAX - 64) return GDN_ERR_ARG;
    if (n_seqs == 0 || n_heads == 0 || n_q == 0) return GDN_OK;
    if ((long long)(n_heads / n_heads_kv) * n_q > INT_MAX - 64) return GDN_ERR_ARG;
    const unsigned long long elt = dtype == GDN_DTYPE_F32 ? 4 : 2, out_elt = out_dtype == GDN_DTYPE_F32 ? 4 : 2;

    // sizes and strides
    long long qs[3] = {(long long)n_heads * n_q * head_dim_k, (long long)n_q * head_dim_k, head_dim_k};
    const int qn[3] = {n_seqs, n_heads, n_q};
    unsigned long long q_reach = (unsigned long long)head_dim_k, q_bytes, out_bytes, mask_bytes = 0, rows, x;
    bool q_align = true;
    for (int i = 0; i < 3; ++i) {
        if (q_strides) qs[i] = q_strides[i];
        if (qn[i] <= 1) continue;
        if (qs[i] < 0 || !mul_ok((unsigned long long)(qn[i] - 1), (unsigned long long)qs[i], &x) || x > (1ull << 59))
            return GDN_ERR_ARG;
        q_reach += x;
        q_align &= (unsigned long long)qs[i] * elt % 16 == 0;
    }
    if (!span_bytes(q_reach, elt, &q_bytes) ||
        !mul_ok((unsigned long long)n_seqs * (unsigned long long)n_heads, (unsigned long long)n_q * head_dim_v, &rows) ||
        !span_bytes(rows, out_elt, &out_bytes))
        return GDN_ERR_ARG;
    if (mask && (!mul_ok((unsigned long long)n_seqs * (unsigned long long)n_q,
                         (unsigned long long)max_pages * (unsigned long long)page_size, &x) ||
                 !span_bytes(x, elt, &mask_bytes)))
        return GDN_ERR_ARG;
    Plan plan;
    if (!plan_of(n_seqs, n_heads, n_heads_kv, n_q, head_dim_k, head_dim_v, page_size, max_pages, (int)elt, &plan))
        return GDN_ERR_ARG;
    const unsigned long long table_bytes = 4ull * (unsigned long long)n_seqs * (unsigned long long)max_pages;
    Layout kl, vl;
    int rc = layout_of(cache_strides, n_pages, n_heads_kv, page_size, head_dim_k, elt, &kl);
    if (rc == GDN_OK)
        rc = layout_of(cache_strides ? cache_strides + 3 : nullptr, n_pages, n_heads_kv, page_size, head_dim_v, elt, &vl);
    if (rc != GDN_OK) return rc;
    if (n_pages == 0) kl.bytes = vl.bytes = 0;

    if (!q || !out || !seq_lens || (max_pages > 0 && !page_table) || (n_pages > 0 && (!k_cache || !v_cache)))
        return GDN_ERR_ARG;
    if (!q_align || !aligned(q, 16) || !aligned(out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(page_table, 4) || !aligned(seq_lens, 4) || !aligned(mask, elt))
        return GDN_ERR_ALIGN;
    const Range ro = range_of(out, out_bytes);
    const Range in[] = {range_of(q, q_bytes), range_of(k_cache, kl.bytes), range_of(v_cache, vl.bytes),
                        range_of(page_table, table_bytes), range_of(seq_lens, 4ull * (unsigned)n_seqs),
                        range_of(mask, mask_bytes)};
    for (Range r : in)
        if (overlap(ro, r)) return GDN_ERR_ALIAS;
    if (workspace && plan.bytes) {
        if (workspace_bytes < plan.bytes || !aligned(workspace, 256)) return GDN_ERR_WORKSPACE;
        const Range rw = range_of(workspace, plan.bytes);
        if (overlap(rw, ro)) return GDN_ERR_ALIAS;
        for (Range r : in)
            if (overlap(rw, r)) return GDN_ERR_ALIAS;
    }

    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (max_pages == 0) plan.grid = 1, plan.cluster = 0, plan.bytes = 0;   // every sequence is empty: zeros
    CUtensorMap km{}, vm{};
    if (n_pages > 0 && (!make_map(&km, k_cache, kl, head_dim_k, dtype) || !make_map(&vm, v_cache, vl, head_dim_v, dtype)))
        return GDN_ERR_CUDA;
    Attn a{};
    a.q = q;
    a.mask = mask;
    a.out = out;
    a.table = page_table;
    a.lens = seq_lens;
    a.status = gdn::status_word();
    if (!a.status) return GDN_ERR_CUDA;
    a.q_seq = qs[0];
    a.q_head = qs[1];
    a.q_query = qs[2];
    a.n_seqs = n_seqs;
    a.H = n_heads;
    a.Hkv = n_heads_kv;
    a.n_q = n_q;
    a.R = n_heads / n_heads_kv * n_q;
    a.n_rb = plan.share.units;
    a.blocks = plan.share.blocks;
    a.groups = plan.share.groups;
    a.ring = plan.share.ring;
    a.n_pages = n_pages;
    a.tpp = page_size / kTile;
    a.max_pages = max_pages;
    a.scale = scale;
    a.out_type = out_dtype;
    a.cluster = plan.cluster;
    for (a.cluster_log = 0; (1 << a.cluster_log) < plan.cluster; ++a.cluster_log) {}
    a.rep = n_heads / n_heads_kv;
    a.by_q = Divisor::of(n_q);
    a.by_rb = Divisor::of(plan.share.units);
    a.by_tpp = Divisor::of(page_size / kTile);
    a.by_units = Divisor::of(n_heads_kv * plan.share.units);
    a.causal = causal != 0;
    a.k_order = kl.order;
    a.v_order = vl.order;
    void *ws = workspace;
    bool owned = false;
    if (plan.bytes && !ws) {
        cudaMemPool_t pool = gdn::workspace_pool();
        if (!pool) return GDN_ERR_CUDA;
        if (cudaMallocFromPoolAsync(&ws, plan.bytes, pool, st) != cudaSuccess) return GDN_ERR_NOMEM;
        owned = true;
    }
    a.ws = static_cast<float *>(ws);
    auto launch = [&](auto type) {
        using T = decltype(type);
        switch (head_dim_k) {
            case 64: return launch_attn<T, 64>(head_dim_v, km, vm, a, plan.grid, st);
            case 128: return launch_attn<T, 128>(head_dim_v, km, vm, a, plan.grid, st);
            default: return launch_attn<T, 256>(head_dim_v, km, vm, a, plan.grid, st);
        }
    };
    cudaError_t e = dtype == GDN_DTYPE_F32    ? launch(float())
                    : dtype == GDN_DTYPE_BF16 ? launch(__nv_bfloat16())
                                              : launch(__half());
    if (owned) {
        const cudaError_t f = cudaFreeAsync(ws, st);
        if (e == cudaSuccess) e = f;
    }
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
