// What the kernels of decode attention over the 4-bit cache share: a call, how its
// work is shared out, and the kernel that joins partial results.
#pragma once

#include <cmath>
#include <cstdint>

#include "../../include/gdn.h"
#include "gdn_internal.h"
#include "gdn_kv4.cuh"

namespace gdn {
namespace kv4 {

constexpr int kGrid = 152;             // CTAs: one per SM of the GPU this is written for

struct Attn {
    View c;
    const void *q, *mask;
    void *out;
    float *ws;
    int n_seqs, H, n_q, R, n_rb, W;    // R rows a kv head in n_rb blocks; W runs at most
    int rows, shift;                   // rows of a block; a step of the schedule is 2^shift tokens
    float scale;
    int q_type, out_type;
    bool causal;
    bool alone;                        // a block a unit, and no partial results
};

constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
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

// 2 consecutive outputs
__device__ __forceinline__ void store2(void *out, int type, size_t i, float x, float y) {
    if (type == GDN_DTYPE_F32)
        *reinterpret_cast<float2 *>(static_cast<float *>(out) + i) = make_float2(x, y);
    else if (type == GDN_DTYPE_BF16)
        *reinterpret_cast<__nv_bfloat162 *>(static_cast<__nv_bfloat16 *>(out) + i) = __floats2bfloat162_rn(x, y);
    else
        *reinterpret_cast<__half2 *>(static_cast<__half *>(out) + i) = __floats2half2_rn(x, y);
}

__device__ __forceinline__ int steps_of(const Attn &a, int len) { return (len + (1 << a.shift) - 1) >> a.shift; }

// Steps of all units of sequence b.  Whole-warp: their total over the sequences
// before `end`, and the sequence that step x lies in with the steps before it.
__device__ __forceinline__ int steps_at(const Attn &a, int b, int units) {
    return b < a.n_seqs ? steps_of(a, length(a.c, b)) * units : 0;
}
__device__ __forceinline__ int steps_before(const Attn &a, int units, int end, int lane) {
    int n = 0;
    for (int b = lane; b < end; b += 32) n += steps_at(a, b, units);
    return __reduce_add_sync(0xffffffffu, n);
}
__device__ __forceinline__ int find_step(const Attn &a, int units, int x, int lane, int *before) {
    int done = 0;
    for (int base = 0;; base += 32) {
        const int n = steps_at(a, base + lane, units);
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

// Floats of a partial result: [rows][DV] outputs, [rows] maxima, [rows] sums.
template <int DV> __device__ __forceinline__ size_t partial(int rows) { return (size_t)rows * (DV + 2); }

// A walk over a run: the unit and the step that it has reached.
struct Cursor {
    int left;                          // steps of the run from here on
    int b, u, j, n, len;               // sequence, unit of it, step of the unit, steps of a unit, tokens
    __device__ __forceinline__ int batch(int U) const { return min(min(U, n - j), left); }
    __device__ __forceinline__ void step(const Attn &a, int units, int k) {
        left -= k;
        j += k;
        if (j < n) return;
        j = 0;
        if (++u == units) {
            u = 0;
            if (left > 0) {            // the next sequence that holds anything
                do {
                    len = length(a.c, ++b);
                    n = steps_of(a, len);
                } while (n == 0);
            }
        }
    }
};

// The walk over run w of the call, from its first step (whole warp).
__device__ __forceinline__ Cursor run_of_call(const Attn &a, int units, int T, int W, int w, int lane) {
    Cursor c;
    const int at = run_begin(T, W, w);
    int before;
    c.left = run_begin(T, W, w + 1) - at;
    c.b = find_step(a, units, at, lane, &before);
    c.len = length(a.c, c.b);
    c.n = steps_of(a, c.len);
    c.u = (at - before) / c.n;
    c.j = at - before - c.u * c.n;
    return c;
}

// Joins the partial results of the rows that several runs share.  A block has
// `rpb` rows, a warp each.  A warp reads the maxima and sums of up to 32 parts at
// once, so their weights are known before the outputs are read, and those loads
// do not wait for one another.  A row of more parts is left to the whole block.
constexpr int kJoinWarps = 8;
template <int DV>
struct Join {
    static constexpr int V = DV == 64 ? 2 : 4, C = DV == 256 ? 2 : 1;   // columns of a lane: C times V
    float x[C * V];
    float M, L;
    // parts first, first + step, ... below n of a row; part 0 is in its run's slot 1
    __device__ __forceinline__ void parts(const float *ws, int rows, int w0, int n, int local, int first,
                                          int step, int lane) {
        M = -INFINITY;
        L = 0.f;
#pragma unroll
        for (int e = 0; e < C * V; ++e) x[e] = 0.f;
        for (int p0 = first; p0 < n; p0 += 32 * step) {
            const int mine = p0 + lane * step, cnt = min(32, (n - p0 + step - 1) / step);
            const float *at = ws + (size_t)partial_slot(w0 + mine, mine == 0) * partial<DV>(rows);
            float m = -INFINITY, l = 0.f;
            if (mine < n) {
                m = __ldcg(at + rows * DV + local);
                l = __ldcg(at + rows * (DV + 1) + local);
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
                    const float *row = ws + (size_t)partial_slot(w0 + p, p == 0) * partial<DV>(rows) + local * DV;
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        if constexpr (V == 2) {
                            const float2 y = __ldcg(reinterpret_cast<const float2 *>(row) + lane);
                            v[i][0] = y.x; v[i][1] = y.y;
                        } else {
                            const float4 y = __ldcg(reinterpret_cast<const float4 *>(row + 128 * c) + lane);
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

template <int DV>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const Attn a, int rpb, int n_rows) {
    __shared__ int s_w0[kJoinWarps], s_n[kJoinWarps];
    __shared__ float s_m[kJoinWarps], s_l[kJoinWarps], s_x[kJoinWarps][DV];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int units = a.c.Hkv * a.n_rb;
    const int T = steps_before(a, units, a.n_seqs, lane), W = min(a.W, T);
    auto place = [&](int r, int &local) {              // where a row's output goes
        const int unit = r / a.R, row = r - unit * a.R, b = unit / a.c.Hkv, hk = unit - b * a.c.Hkv;
        local = row % a.rows;
        return (((size_t)b * a.n_q + row % a.n_q) * a.H + hk * (a.H / a.c.Hkv) + row / a.n_q) * DV;
    };
    const int r0 = blockIdx.x * rpb, r = r0 + warp;
    int w0 = 0, n = -1;                                // runs that share the row; -1: none of ours
    if (warp < rpb && r < n_rows) {
        const int unit = r / a.R, row = r - unit * a.R, b = unit / a.c.Hkv, hk = unit - b * a.c.Hkv;
        const int tiles = steps_of(a, length(a.c, b));
        n = 0;
        if (tiles > 0) {
            const int first = steps_before(a, units, b, lane) + (hk * a.n_rb + row / a.rows) * tiles;
            w0 = run_of(T, W, first);
            n = run_of(T, W, first + tiles - 1) - w0 + 1;
        }
    }
    if (lane == 0) {
        s_w0[warp] = w0;
        s_n[warp] = n;
    }
    // the attention kernel's results; every block waits, so that this grid never
    // ends before that one
    asm volatile("griddepcontrol.wait;" ::: "memory");
    Join<DV> join;
    int local;
    if (n >= 0 && n != 1 && n <= 32) {                 // (one run had it all: written; none: zeros)
        const size_t at = place(r, local);
        join.parts(a.ws, a.rows, w0, n, local, 0, 1, lane);
        join.store(a, at, lane);
    }
    __syncthreads();
    for (int i = 0; i < rpb; ++i) {
        if (s_n[i] <= 32) continue;
        const size_t at = place(r0 + i, local);
        join.parts(a.ws, a.rows, s_w0[i], s_n[i], local, warp, kJoinWarps, lane);
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
            for (int k = 0; k < kJoinWarps; ++k) top = fmaxf(top, s_m[k]);
            const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
            for (int e = 0; e < join.C * join.V; ++e) join.x[e] = 0.f;
#pragma unroll
            for (int k = 0; k < kJoinWarps; ++k) {
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

// Launches the join as a programmatic dependent of the attention kernel before it.
// Its blocks start as that kernel's end (no earlier trigger: blocks that only wait
// would gather on the first SM that has room, and stay there).  2 x 16/4 x (100003,
// 50001) x 128: 52 us triggered at the kernel's start, 42 at its end, 44 as a plain
// launch.
template <int DV>
cudaError_t launch_join(const Attn &a, cudaStream_t stream) {
    // few rows: a block each, so that long rows are shared out; many: a warp each
    const int n_rows = a.n_seqs * a.c.Hkv * a.R;
    const int rpb = (int)(n_rows >= 2 * kGrid * kJoinWarps ? kJoinWarps : (n_rows + 2 * kGrid - 1) / (2 * kGrid));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(((unsigned)n_rows + rpb - 1) / rpb);
    cfg.blockDim = dim3(kJoinWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, join_kernel<DV>, a, rpb, n_rows);
}

// Many rows a kv head (gdn_kv4_rows.cu): blocks of kManyRows rows, steps of 128 tokens.
constexpr int kManyRows = 32;
bool many_rows_ok(int dk, int dv);
cudaError_t launch_many_rows(const Attn &a, cudaStream_t stream);

}  // namespace kv4
}  // namespace gdn
