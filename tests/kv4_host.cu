// The 4-bit cache's index and rounding arithmetic, compiled for the host, so
// that it is tested where there is no GPU (tests/test_kv4_host.py).
#include <cstdint>

#include "../include/gdn.h"
#include "../linear_attention_sequence_gated_gb300/csrc/gdn_kv4.cuh"

extern "C" {

long long kv4_tile_offset(int page, int n_pages, int Hkv, int h, int tpp, int in_page, int bytes) {
    return gdn::kv4::tile_offset(page, n_pages, Hkv, h, tpp, in_page, bytes);
}

// tile, t0, held, then 16 flags: token t0 + i is present
void kv4_place(int raw, int cap, int count, int j, int *out) {
    const gdn::kv4::Place p = gdn::kv4::place_of(raw, cap, count, j);
    out[0] = p.tile;
    out[1] = p.t0;
    out[2] = p.held();
    for (int i = 0; i < 16; ++i) out[3 + i] = p.present(p.t0 + i);
}

void kv4_scale_bytes(const float *a, int n, int wide, int *out) {
    for (int i = 0; i < n; ++i) out[i] = wide ? gdn::kv4::scale_byte(a[i]) : gdn::kv4::scale_byte16(a[i]);
}

// quotients by scale `byte` as the conversion to 4 bits takes them
void kv4_ratios(const float *x, int n, int byte, int wide, float *out) {
    // 16-bit elements: an approximate reciprocal will do, here one that is 2 units off
    const float s = gdn::kv4::scale_value(byte), r = wide ? 1.f / s : 1.f / s * (1.f + 3e-7f);
    for (int i = 0; i < n; ++i) out[i] = wide ? gdn::kv4::ratio32(x[i], r, s) : gdn::kv4::ratio16(x[i], r);
}
int kv4_run_begin(int T, int W, int w) { return gdn::kv4::run_begin(T, W, w); }
int kv4_run_of(int T, int W, int x) { return gdn::kv4::run_of(T, W, x); }
int kv4_partial_slot(int w, int begins_here) { return gdn::kv4::partial_slot(w, begins_here != 0); }

}  // extern "C"
