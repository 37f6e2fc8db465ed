// Pages handed out and taken back on the device (gdn_page_assign, gdn_page_release).
//
// Pages that nobody holds lie on a stack: free[0 .. count).  A step that adds n_b tokens to
// sequence b takes ceil(len_b / page) - ceil((len_b - n_b) / page) pages for it; with the
// exclusive sums p_b of these numbers over the sequences, the k-th page of the step
// (k = p_b + j - held_b for entry j of sequence b's table) is free[count - 1 - k].  Every
// entry and every token's slot follows from the two sums (pages and tokens) alone, so all
// are written at once, by one CTA for a decode step and by the whole GPU for prompts, each CTA with
// the sums of all sequences in shared memory.  Only `count` is both read and written: after a barrier
// in one CTA, by a second kernel where there are more.  Pages go back in one cluster, whose
// CTAs count what they have to push (some entries may name no page) before any pushes.
//
// A decode step moves a few hundred bytes, so the call's time is one launch, the lengths'
// latency, a scan and a dependent load or two: 64 sequences x 8 tokens of 16-token pages take 3.4 us, 131072 tokens and 8192
// pages 5.8, all of them back 5.7 (GPU time of captured calls).
#include <climits>
#include <cstdint>

#include "../../include/gdn.h"
#include "gdn_internal.h"
#include "gdn_kv4.cuh"

namespace gdn {
namespace pages {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kMaxSeqs = 16384;        // the two sums of all sequences lie in shared memory
// Work (tokens and sequences; for a release entries of tables) from which a call takes more than one CTA.  (One and more, us:
// 64 sequences x 64 tokens 4.8 and 5.1, x 128 6.3 and 5.4, x 512 14 and 5.6, 1 x 65536 24 and 5.2, 4096 x 1 12.3 and 9.3;
// their 2048 pages back 5.5 in one, 4096 6.6 and 5.2, 8192 9.5 and 5.7.)
constexpr long long kManyItems = 4096;
constexpr int kGrid = 304;             // CTAs at most, two per SM of the GPU this is written for
constexpr int kCluster = 8;            // the largest portable size

struct Step {
    int *table;                        // (n_seqs, max_pages)
    const int *lens, *counts;          // lengths with the step's tokens; tokens each, or NULL: n_new
    const int *free;                   // the stack, with room for n_pages entries
    int *count;
    int *slots, *positions, *offsets;
    int *status;
    int n_seqs, n_new, n_tokens, page, max_pages, n_pages;
    Divisor by_page;
    bool packed;
};

struct Release {
    const int *table, *from, *to;
    int *free, *count, *status;
    int n_seqs, page, max_pages, n_pages;
};

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int cluster_rank() {
    int r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ int cluster_size() {
    int r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ int peer_int(const int *p, int rank) {
    const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p));
    int x;
    asm volatile("{\n\t.reg .u32 r;\n\tmapa.shared::cluster.u32 r, %1, %2;\n\tld.shared::cluster.s32 %0, [r];\n\t}"
                 : "=r"(x) : "r"(a), "r"(rank) : "memory");
    return x;
}

// Exclusive sum of x over the block's threads, and the total; `part` is kWarps + 1 ints of
// shared memory, free again when every thread has passed the next barrier.
__device__ __forceinline__ int block_scan(int x, int *part, int *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += o;
    }
    if (lane == 31) part[warp] = incl;
    __syncthreads();
    int before = lane < kWarps ? part[lane] : 0;
    const int all = __reduce_add_sync(0xffffffffu, before);
    before = __reduce_add_sync(0xffffffffu, lane < warp ? before : 0);
    *total = all;
    return before + incl - x;
}

// The last of the n + 1 ascending values sum[0 .. n] (sum[0] = 0) that is at most x, of equal ones
// the last below n: the sequence that item x < sum[n] belongs to.
__device__ __forceinline__ int owner(const int *sum, int n, int x) {
    int lo = 0, hi = n;                // sum[lo] <= x < sum[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sum[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ int pages_of(int tokens, int page) { return tokens > 0 ? (tokens - 1) / page + 1 : 0; }

// What a step does to a sequence.
struct Seq {
    int first, n;                      // position of its first new token (may be negative), new tokens
    int held, after;                   // pages before and with them
};
__device__ __forceinline__ Seq seq_of(const Step &s, int b, bool *past) {
    const int raw = max(s.lens[b], 0), cap = s.max_pages * s.page;
    Seq q;
    q.n = s.counts ? min(max(s.counts[b], 0), s.n_new) : s.n_new;
    q.first = raw - q.n;
    q.after = pages_of(min(raw, cap), s.page);
    q.held = min(pages_of(q.first, s.page), q.after);
    *past = raw > cap || (s.counts && s.counts[b] > s.n_new);
    return q;
}

__global__ void __launch_bounds__(kThreads) assign_kernel(const Step s) {
    extern __shared__ int sums[];      // [n_seqs + 1] tokens, [n_seqs + 1] pages
    __shared__ int part[2][2][kWarps];
    int *tok = sums, *pg = sums + s.n_seqs + 1;
    kv4::after_the_kernel_before();
    const int tid = threadIdx.x;
    const int raw_count = *s.count;
    bool bad = raw_count < 0 || raw_count > s.n_pages;
    const int count = min(max(raw_count, 0), s.n_pages);
    int tokens = 0, taken = 0;
    for (int base = 0, turn = 0; base < s.n_seqs; base += kThreads, turn ^= 1) {
        const int b = base + tid;
        Seq q = {0, 0, 0, 0};
        if (b < s.n_seqs) {
            bool past;
            q = seq_of(s, b, &past);
            bad |= past;
        }
        int all_tokens, all_pages;
        const int t = block_scan(q.n, part[turn][0], &all_tokens);
        const int p = block_scan(q.after - q.held, part[turn][1], &all_pages);
        if (b < s.n_seqs) {
            tok[b] = tokens + t;
            pg[b] = taken + p;
        }
        tokens += all_tokens;
        taken += all_pages;
    }
    if (tid == 0) {
        tok[s.n_seqs] = tokens;
        pg[s.n_seqs] = taken;
    }
    __syncthreads();
    const int step = gridDim.x * kThreads, me = blockIdx.x * kThreads + tid;
    // the k-th page of the step
    auto page_at = [&](int k) { return k < count ? s.free[count - 1 - k] : -1; };
    bad |= taken > count;
    for (int k = me; k < taken; k += step) {
        const int b = owner(pg, s.n_seqs, k);
        bool past;
        s.table[(size_t)b * s.max_pages + seq_of(s, b, &past).held + k - pg[b]] = page_at(k);
    }
    const int items = s.packed ? s.n_tokens : s.n_seqs * s.n_new;
    if (s.packed) {
        bad |= tokens > s.n_tokens;
        for (int b = me; b <= s.n_seqs; b += step) s.offsets[b] = tok[b];
    }
    // A warp's tokens lie together, a thread's 32 apart, mostly of one sequence.
    const int each = ((items + step - 1) / step) * 32, begin = (me >> 5) * each, lane = tid & 31;
    const int end = min(begin + each, items);
    int b = -1, next = 0, base = 0;    // the sequence of token i, where the one after it begins, and it
    Seq q = {0, 0, 0, 0};
    for (int i = begin + lane; i < end; i += 32) {
        if (b < 0 || i >= next) {
            bool past;
            if (s.packed) {
                b = i < tokens ? owner(tok, s.n_seqs, i) : s.n_seqs;
                base = tok[b];
                next = b < s.n_seqs ? tok[b + 1] : items;
            } else {
                b = i / s.n_new;
                base = b * s.n_new;
                next = base + s.n_new;
            }
            q = {0, 0, 0, 0};
            if (b < s.n_seqs) q = seq_of(s, b, &past);
        }
        const int p = i - base < q.n ? q.first + i - base : -1;
        const int j = p < 0 ? s.max_pages : s.by_page.into(p);
        int slot = -1, pos = 0;
        if (j < s.max_pages) {
            const int page = j < q.held ? s.table[(size_t)b * s.max_pages + j] : page_at(pg[b] + j - q.held);
            pos = p;
            if ((unsigned)page < (unsigned)s.n_pages) slot = page * s.page + p - j * s.page;
            else bad = true;
        }
        s.slots[i] = slot;
        if (s.positions) s.positions[i] = pos;
    }
    if (bad) *s.status = GDN_ERR_PAGE;
    if (gridDim.x == 1) {
        __syncthreads();               // every thread has read the count
        if (tid == 0) *s.count = max(count - taken, 0);
    }
}

// The count after a step of more than one CTA.
__global__ void __launch_bounds__(kThreads) count_kernel(const Step s) {
    __shared__ int part[kWarps];
    kv4::after_the_kernel_before();
    int n = 0, taken;
    for (int b = threadIdx.x; b < s.n_seqs; b += kThreads) {
        bool past;
        const Seq q = seq_of(s, b, &past);
        n += q.after - q.held;
    }
    block_scan(n, part, &taken);
    if (threadIdx.x == 0) *s.count = max(min(max(*s.count, 0), s.n_pages) - taken, 0);
}

// A thread takes kRun neighbouring entries of all that go back, in the order in which an assign took them.
constexpr int kRun = 8;
__global__ void __launch_bounds__(kThreads) release_kernel(const Release s) {
    extern __shared__ int sums[];      // [n_seqs + 1] pages given back before a sequence's, [n_seqs] its first
    __shared__ int part[2][kWarps];
    __shared__ int mine;
    int *pg = sums, *first = sums + s.n_seqs + 1;
    kv4::after_the_kernel_before();
    const int tid = threadIdx.x;
    const int raw_count = *s.count, cap = s.max_pages * s.page;
    bool bad = raw_count < 0 || raw_count > s.n_pages;
    const int count = min(max(raw_count, 0), s.n_pages);
    int given = 0;
    for (int base = 0, turn = 0; base < s.n_seqs; base += kThreads, turn ^= 1) {
        const int b = base + tid;
        int n = 0, to = 0, all;
        if (b < s.n_seqs) {
            const int len = s.from[b];
            const int from = pages_of(min(len, cap), s.page);
            to = s.to ? min(pages_of(min(s.to[b], cap), s.page), from) : 0;
            n = from - to;
            bad |= len > cap;
        }
        const int p = block_scan(n, part[turn], &all);
        if (b < s.n_seqs) {
            pg[b] = given + p;
            first[b] = to;
        }
        given += all;
    }
    if (tid == 0) pg[s.n_seqs] = given;
    __syncthreads();
    // a contiguous share of the entries; those that name no page (the stack had run out) are left out
    const int rank = cluster_rank(), size = cluster_size();
    const int lo = (int)((long long)given * rank / size), hi = (int)((long long)given * (rank + 1) / size);
    auto load = [&](int k0, int (&page)[kRun]) {
        int n = 0;
        int b = k0 < hi ? owner(pg, s.n_seqs, k0) : 0;
#pragma unroll
        for (int u = 0; u < kRun; ++u) {
            const int k = k0 + u;
            page[u] = -1;
            if (k < hi) {
                while (k >= pg[b + 1]) ++b;
                page[u] = s.table[(size_t)b * s.max_pages + first[b] + k - pg[b]];
            }
        }
#pragma unroll
        for (int u = 0; u < kRun; ++u) {
            if ((unsigned)page[u] >= (unsigned)s.n_pages) page[u] = -1;
            n += page[u] >= 0;
        }
        return n;
    };
    constexpr int kBatch = kThreads * kRun;
    int page[kRun], n = 0, held = 0, all;
    for (int base = lo; base < hi; base += kBatch) held += n = load(base + tid * kRun, page);
    block_scan(held, part[0], &all);
    if (tid == 0) mine = all;
    cluster_sync();
    int before = 0;
    all = 0;
    for (int r = 0; r < size; ++r) {
        const int x = peer_int(&mine, r);
        if (r < rank) before += x;
        all += x;
    }
    cluster_sync();                    // every thread has read the count and its peers' shares
    // (64 bits: the stack and the entries may be 2^31 - 1 each)
    const long long full = (long long)count + all;
    bad |= all != given || full > s.n_pages;
    for (int base = lo, turn = 1; base < hi; base += kBatch, turn ^= 1) {
        if (hi - lo > kBatch) n = load(base + tid * kRun, page);       // (else they are here already)
        int sum;
        long long at = full - 1 - before - block_scan(n, part[turn], &sum);
#pragma unroll
        for (int u = 0; u < kRun; ++u)
            if (page[u] >= 0) {
                if (at < s.n_pages) s.free[at] = page[u];
                --at;
            }
        before += sum;
    }
    if (bad) *s.status = GDN_ERR_PAGE;
    if (rank == 0 && tid == 0) *s.count = (int)min(full, (long long)s.n_pages);
}

cudaError_t launch_cluster(const Release &args, long long items, size_t smem, cudaStream_t stream) {
    cudaLaunchAttribute attr[2];
    const unsigned cl = items >= kManyItems ? kCluster : 1;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cl;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(cl);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, release_kernel, args);
}

// The checks that both calls share; fills the status word's address.
int check(const int *table, const int *free_pages, const int *count, int n_seqs, int page, int max_pages,
          int n_pages) {
    using namespace host;
    if (n_seqs < 0 || max_pages < 0 || n_pages < 0) return GDN_ERR_ARG;
    if (page < 1 || n_seqs > kMaxSeqs) return GDN_ERR_SHAPE;
    if ((long long)max_pages * page > INT_MAX || (long long)n_pages * page > INT_MAX ||
        (long long)n_seqs * max_pages > INT_MAX - kGrid * kThreads)       // (indices step past the end)
        return GDN_ERR_ARG;
    if (n_seqs == 0) return GDN_OK;
    if ((max_pages > 0 && !table) || (n_pages > 0 && !free_pages) || !count) return GDN_ERR_ARG;
    if (!aligned(table, 4) || !aligned(free_pages, 4) || !aligned(count, 4)) return GDN_ERR_ALIGN;
    return GDN_OK;
}

int opt_in() {                         // shared memory for the sums of kMaxSeqs sequences
    static PerDeviceOnce setup;
    return setup.run([] {
        cudaError_t e = cudaFuncSetAttribute(assign_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             2 * (kMaxSeqs + 1) * (int)sizeof(int));
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(release_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (2 * kMaxSeqs + 1) * (int)sizeof(int));
        return e;
    }) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace
}  // namespace pages
}  // namespace gdn

extern "C" {

int gdn_page_assign(int *page_table, const int *seq_lens, const int *new_lens, const int *free_pages,
                    int *free_count, int *slots, int *positions, int *token_offsets, int n_seqs, int n_new, int n_tokens,
                    int page_size, int max_pages, int n_pages, gdn_stream_t stream) {
    using namespace gdn::host;
    using namespace gdn::pages;
    if (n_new < 0 || n_tokens < 0) return GDN_ERR_ARG;
    const int rc = check(page_table, free_pages, free_count, n_seqs, page_size, max_pages, n_pages);
    if (rc != GDN_OK) return rc;
    if ((long long)n_seqs * n_new > INT_MAX) return GDN_ERR_ARG;
    const bool packed = token_offsets != nullptr;
    const long long items = packed ? n_tokens : (long long)n_seqs * n_new;
    if (items > INT_MAX - kGrid * kThreads) return GDN_ERR_ARG;
    if (n_seqs == 0 && items == 0 && !packed) return GDN_OK;
    if ((n_seqs > 0 && !seq_lens) || (items > 0 && !slots) || !free_count) return GDN_ERR_ARG;
    if (!aligned(seq_lens, 4) || !aligned(new_lens, 4) || !aligned(slots, 4) || !aligned(positions, 4) ||
        !aligned(token_offsets, 4) || !aligned(free_count, 4))
        return GDN_ERR_ALIGN;
    const unsigned long long lens = 4ull * (unsigned)n_seqs;
    const Range out[] = {range_of(page_table, 4ull * (unsigned long long)n_seqs * (unsigned)max_pages),
                         range_of(free_count, 4), range_of(slots, 4ull * (unsigned long long)items),
                         range_of(positions, 4ull * (unsigned long long)items),
                         range_of(token_offsets, packed ? lens + 4 : 0)};
    const Range in[] = {range_of(seq_lens, lens), range_of(new_lens, lens),
                        range_of(free_pages, 4ull * (unsigned)n_pages)};
    for (int i = 0; i < 5; ++i) {
        for (Range r : in)
            if (overlap(out[i], r)) return GDN_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return GDN_ERR_ALIAS;
    }
    int *status = gdn::status_word();
    if (!status || opt_in() != GDN_OK) return GDN_ERR_CUDA;
    const Step s{page_table, seq_lens, new_lens, free_pages, free_count, slots, positions, token_offsets, status,
                 n_seqs, n_new, n_tokens, page_size, max_pages, n_pages, gdn::Divisor::of(page_size), packed};
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    // a thread takes two tokens or more before there are more CTAs
    const long long work = items + n_seqs;
    const unsigned grid = work < kManyItems ? 1u : (unsigned)(work / (2 * kThreads) < kGrid ? work / (2 * kThreads) : kGrid);
    cudaError_t e = gdn::kv4::launch_early(assign_kernel, dim3(grid), kThreads, 2 * ((size_t)n_seqs + 1) * sizeof(int), st, s);
    if (e == cudaSuccess && grid > 1) e = gdn::kv4::launch_early(count_kernel, dim3(1), kThreads, 0, st, s);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

int gdn_page_release(const int *page_table, const int *from_lens, const int *to_lens, int *free_pages,
                     int *free_count, int n_seqs, int page_size, int max_pages, int n_pages, gdn_stream_t stream) {
    using namespace gdn::host;
    using namespace gdn::pages;
    const int rc = check(page_table, free_pages, free_count, n_seqs, page_size, max_pages, n_pages);
    if (rc != GDN_OK || n_seqs == 0) return rc;
    if (!from_lens) return GDN_ERR_ARG;
    if (!aligned(from_lens, 4) || !aligned(to_lens, 4)) return GDN_ERR_ALIGN;
    const unsigned long long lens = 4ull * (unsigned)n_seqs;
    const Range out[] = {range_of(free_pages, 4ull * (unsigned)n_pages), range_of(free_count, 4)};
    if (overlap(out[0], out[1])) return GDN_ERR_ALIAS;
    for (Range r : {range_of(page_table, 4ull * (unsigned long long)n_seqs * (unsigned)max_pages),
                    range_of(from_lens, lens), range_of(to_lens, lens)})
        if (overlap(out[0], r) || overlap(out[1], r)) return GDN_ERR_ALIAS;
    int *status = gdn::status_word();
    if (!status || opt_in() != GDN_OK) return GDN_ERR_CUDA;
    const Release s{page_table, from_lens, to_lens, free_pages, free_count, status, n_seqs, page_size, max_pages,
                    n_pages};
    return launch_cluster(s, (long long)n_seqs * max_pages, (2 * (size_t)n_seqs + 1) * sizeof(int),
                          reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
