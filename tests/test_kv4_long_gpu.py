"""GPU tests of decode attention over the 4-bit cache where each warp walks
hundreds of steps: as many (sequence, kv head) units as the GPU has warps at
work, each of up to 512 steps.

The tokens are few: the entries of a sequence's page table name the same pages
again and again, two of them in its first half and two others in its second, so
that a step that weighs early tokens otherwise than late ones shows.  The float64
reference then counts each token as often as the table names it.

Metric and bound as in test_kv4_attn_gpu.py: max |gpu - oracle| / RMS(oracle) <=
1e-4 for fp32 outputs.  What runs of this length add to its account: the sum of
the weights and the output take one fp32 rounding a step, half a unit of 2^-23 of
what they are, 512 x 2^-24 = 3e-5 in all if every one went one way.  Scores near 40
(every key has the same first 16 elements) are off by up to 16 units of 2^-23 of
40, 8e-5, but by the same amount for the part that all tokens share, which is
nearly all of it and cancels; what differs are scores of a few units, as there.
"""
import numpy as np
import pytest
import torch

import linear_attention_sequence_gated_gb300 as gdn
import oracle
from oracle import kv4

pytestmark = pytest.mark.gpu

TOL = 1e-4
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
PAGE, PAGES = 256, 4                  # tokens a page; pages there are


@pytest.fixture(scope="module", autouse=True)
def built():
    from linear_attention_sequence_gated_gb300 import _build
    _build.build()


class Long:
    def __init__(self, dk, dv, dtype, rep, B, n, offset, seed=0):
        Hkv = 8
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        f = dict(generator=gen, device="cuda")
        self.cache = gdn.kv4_cache(PAGES, Hkv, PAGE, dk, dv)
        k = torch.randn((1, Hkv, PAGES * PAGE, dk), **f)
        v = torch.randn((1, Hkv, PAGES * PAGE, dv), **f)
        k[..., :16] = 3.0
        whole = torch.tensor([PAGES * PAGE], dtype=torch.int32, device="cuda")
        gdn.kv4_write(k, v, self.cache, torch.arange(PAGES, dtype=torch.int32, device="cuda").reshape(1, PAGES), whole)
        self.k, self.v = (torch.tensor(kv4.kept(x.double().cpu().numpy()), device="cuda")[0] for x in (k, v))
        assert (self.k[..., :16] == 3.0).all()
        slots = n // PAGE
        entry = np.arange(slots)
        entry = np.where(entry < slots // 2, entry % 2, 2 + entry % 2)
        self.table = torch.tensor(np.tile(entry, (B, 1)), dtype=torch.int32, device="cuda")
        lens = n - np.arange(B) % 5 * 13                       # the last tile, step and page in full and in part
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.seen = np.zeros((B, PAGES, PAGE))                 # how often each token is one of a sequence's
        for e, p in enumerate(entry):
            self.seen[:, p] += np.arange(PAGE)[None] < np.clip(lens - e * PAGE, 0, PAGE)[:, None]
        self.dv, self.entry = dv, entry
        q = torch.randn((B, Hkv * rep, 1, dk), **f)
        scale = dk ** -0.5
        if offset:
            q[..., :16] = (offset + 5 * torch.rand((B, Hkv * rep, 1, 1), **f)) / (48 * scale)
        self.q = q.to(DTYPES[dtype])
        self.add = torch.randn((PAGES, PAGE), **f).to(DTYPES[dtype])      # a mask's value for each token

    def mask(self):
        row = self.add[torch.tensor(self.entry, device="cuda")].reshape(-1)
        return row.expand(self.q.shape[0], 1, 1, -1).contiguous()

    def want(self, masked, v):
        B, H, _, dk = self.q.shape
        Hkv = self.k.shape[0]
        q = self.q.double().reshape(B, Hkv, H // Hkv, dk)
        s = torch.einsum("bgrd,gnd->bgrn", q, self.k) * float(np.float32(dk ** -0.5))
        if masked:
            s = s + self.add.double().reshape(-1)
        w = torch.exp(s - s.amax(-1, keepdim=True)) * torch.tensor(self.seen, device="cuda").reshape(B, 1, 1, -1)
        return (torch.einsum("bgrn,gnd->bgrd", w, v) / w.sum(-1, keepdim=True)).reshape(B, 1, H, self.dv)

    def check(self, masked=False, out_dtype=None):
        got = gdn.flash_attn_kv4(self.q, self.cache, self.table, self.lens, self.dv, self.mask() if masked else None,
                                 out_dtype=out_dtype)
        ref = self.want(masked, self.v)
        torch.cuda.synchronize()
        assert gdn.device_status() == gdn.OK and torch.isfinite(got).all()
        if got.dtype == torch.float32:
            assert oracle.parity_error(got.double().cpu().numpy(), ref.cpu().numpy()) <= TOL
        else:
            off = TOL * ref.square().mean().sqrt() + 2.0 ** -11 * self.want(masked, self.v.abs())
            step = torch.finfo(got.dtype).eps / 2
            assert ((got.double() - ref).abs() <= off + step * (ref.abs() + off) + 2.0 ** -25).all()


# 12 warps an SM take steps of 64 tokens at widths up to 128, 8 warps steps of 32 at others
def shape(dk, dv):
    return (228, 32768) if max(dk, dv) <= 128 else (152, 16384)


@pytest.mark.parametrize("offset", [0, 40])
@pytest.mark.parametrize("dtype,rep,out", [("bf16", 1, None), ("f16", 8, None), ("f32", 2, None), ("f16", 4, "f16"),
                                           ("bf16", 8, "bf16")])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (64, 256), (256, 256)])
def test_runs_of_512_steps(dk, dv, dtype, rep, out, offset):
    B, n = shape(dk, dv)
    Long(dk, dv, dtype, rep, B, n, offset, seed=dk + dv + rep).check(out_dtype=out and DTYPES[out])


@pytest.mark.parametrize("dk,dv", [(128, 128), (256, 128)])
def test_runs_of_512_steps_with_a_mask(dk, dv):
    B, n = shape(dk, dv)
    Long(dk, dv, "bf16", 2, B, n, 40, seed=dk).check(masked=True)


@pytest.mark.parametrize("dk,dv", [(64, 128), (128, 64), (256, 64), (128, 256), (256, 256)])
@pytest.mark.parametrize("dtype,rep", [("bf16", 3), ("f32", 9)])
def test_runs_over_parts_of_units(dk, dv, dtype, rep):
    """40 sequences: a unit lies in several runs of about 20 steps, rings wrap, and the join adds them up."""
    Long(dk, dv, dtype, rep, 40, 8192 if max(dk, dv) <= 128 else 4096, 20, seed=dk + dv).check()
