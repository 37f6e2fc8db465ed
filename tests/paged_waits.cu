// The paged attention's kernel (f16 rows, keys of width 64) with its waits looked at: which uses of the ring's stages the
// warps that filled them have seen land; and with one warp of one CTA acting, from a wait on that a test names, as if its
// waits had run out.  No copy is left out, so nothing hangs and no wait runs long.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../include/gdn.h"
#include "../linear_attention_sequence_gated_gb300/csrc/gdn_internal.h"
#include "../linear_attention_sequence_gated_gb300/csrc/gdn_kv4.cuh"
#include "../linear_attention_sequence_gated_gb300/csrc/gdn_ptx.cuh"

constexpr int kSlots = 1 << 15;        // 8-byte places of shared memory
struct Seen {
    int cta;                           // the one that is looked at
    int loser, lives, lost;            // its warp that gives up (-1: none), the waits that this one lives through, whether it did
    int waits[32];                     // of each of its warps
    int filled[kSlots], landed[kSlots];    // of the barrier at each place: uses, and the last that its filler saw land
};
__device__ Seen g_seen;

namespace gdn {
namespace ptx {

__device__ __forceinline__ void expect_and_count(uint64_t *bar, uint32_t bytes) {
    if ((int)blockIdx.x == g_seen.cta) ++g_seen.filled[smem_u32(bar) / 8 % kSlots];
    mbar_arrive_expect_tx(bar, bytes);
}
__device__ __forceinline__ bool wait_and_look(uint64_t *bar, uint32_t parity, const volatile int *abort) {
    const int warp = threadIdx.x >> 5;
    if ((int)blockIdx.x == g_seen.cta) {
        const int n = *(volatile int *)&g_seen.waits[warp];
        __syncwarp();
        if ((threadIdx.x & 31) == 0) *(volatile int *)&g_seen.waits[warp] = n + 1;
        __syncwarp();
        // (never a filling warp's wait for its own copies)
        if (warp == g_seen.loser && n >= g_seen.lives &&
            !(threadIdx.x + 128 >= blockDim.x && g_seen.filled[smem_u32(bar) / 8 % kSlots] > 0)) {
            g_seen.lost = 1;
            return false;
        }
    }
    const bool came = mbar_wait(bar, parity, abort);
    if ((int)blockIdx.x == g_seen.cta && (threadIdx.x & 31) == 0 && threadIdx.x + 128 >= blockDim.x) {
        const int at = smem_u32(bar) / 8 % kSlots, n = g_seen.filled[at];     // (0: not a barrier that copies complete)
        if (came && n > 0 && parity == (uint32_t)((n - 1) & 1)) g_seen.landed[at] = n;
    }
    return came;
}

}  // namespace ptx
}  // namespace gdn

#define mbar_wait wait_and_look
#define mbar_arrive_expect_tx expect_and_count
#define GDN_PAGED_ATTN_T __half
#define GDN_PAGED_ATTN_DK 64
#include "../linear_attention_sequence_gated_gb300/csrc/gdn_paged_attn.cuh"
#undef mbar_wait
#undef mbar_arrive_expect_tx
namespace gdn {
namespace paged {                      // the library's own
#define OTHER(T, DK) \
    extern template cudaError_t launch_attn<T, DK>(int, const CUtensorMap &, const CUtensorMap &, const Attn &, int, cudaStream_t)
OTHER(__half, 128);
OTHER(__half, 256);
OTHER(__nv_bfloat16, 64);
OTHER(__nv_bfloat16, 128);
OTHER(__nv_bfloat16, 256);
OTHER(float, 64);
OTHER(float, 128);
OTHER(float, 256);
}  // namespace paged
}  // namespace gdn
#include "../linear_attention_sequence_gated_gb300/csrc/gdn_paged_attn.cu"

static Seen h_seen;
extern "C" int look_at(int cta, int loser, int lives) {
    h_seen = Seen{};
    h_seen.cta = cta;
    h_seen.loser = loser;
    h_seen.lives = lives;
    return (int)cudaMemcpyToSymbol(g_seen, &h_seen, sizeof(h_seen));
}
extern "C" int was_lost() {
    return cudaMemcpyFromSymbol(&h_seen, g_seen, sizeof(h_seen)) == cudaSuccess ? h_seen.lost : -1;
}
// Stages that were filled, and those of them whose last use their filler did not see land.
extern "C" int stages(int *unseen) {
    if (cudaMemcpyFromSymbol(&h_seen, g_seen, sizeof(h_seen)) != cudaSuccess) return -1;
    int n = *unseen = 0;
    for (int i = 0; i < kSlots; ++i) {
        n += h_seen.filled[i] > 0;
        *unseen += h_seen.filled[i] != h_seen.landed[i];
    }
    return n;
}
