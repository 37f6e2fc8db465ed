// Host arithmetic of the paged attention, for tests without a GPU.
#include "../linear_attention_sequence_gated_gb300/csrc/gdn_paged_attn.cuh"

extern "C" void paged_share(int dk, int dv, int elt, int R, int *out) {
    using namespace gdn::paged;
    const Share s = share_of(dk, dv, elt, R);
    const Room r = room_of(dk, dv, elt, s.warps, s.most);
    const int x[8] = {s.warps, s.most, s.blocks, s.groups, s.units, s.ring, r.pool, s.blocks * r.q_block};
    for (int i = 0; i < 8; ++i) out[i] = x[i];
}

// The quotients as the device takes them: the upper half of a 32 x 32-bit product, shifted.
extern "C" void paged_quotients(int d, const int *x, int n, int *out) {
    const gdn::Divisor v = gdn::Divisor::of(d);
    for (int i = 0; i < n; ++i)
        out[i] = v.l ? (int)(((unsigned long long)(unsigned)x[i] * v.m >> 32) >> (v.l - 1)) : x[i];
}
