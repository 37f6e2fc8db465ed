"""GPU tests of the waits in the paged attention, with a build of its kernel that counts them (tests/paged_waits.cu)."""
import ctypes
import os
import subprocess

import pytest
import torch

import linear_attention_sequence_gated_gb300 as gdn
from linear_attention_sequence_gated_gb300 import _build
from test_paged_attn_gpu import Case

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def X(tmp_path_factory):
    lib = _build.build()
    so = str(tmp_path_factory.mktemp("paged") / "paged_waits.so")
    subprocess.check_call([_build.nvcc()] + _build.ARCH + ["-O3", "-std=c++17", "--expt-relaxed-constexpr", "-shared", "-Xcompiler",
                                                          "-fPIC", "-o", so, os.path.join(HERE, "paged_waits.cu"), lib])
    gdn.lib()
    x = ctypes.CDLL(so)
    x.gdn_flash_attn_paged.argtypes = gdn.lib().gdn_flash_attn_paged.argtypes
    return x


def run(X, c):
    B, H, n_q, dk = c.q.shape
    n_pages, Hkv, page, dv = c.vc.shape
    out = torch.zeros((B, n_q, H, dv), device="cuda")
    rc = X.gdn_flash_attn_paged(c.q.data_ptr(), None, c.kc.data_ptr(), c.vc.data_ptr(), None, c.table.data_ptr(),
                                c.lens.data_ptr(), None, out.data_ptr(), B, H, Hkv, n_q, dk, dv, n_pages, page, c.table.shape[1],
                                dk ** -0.5, 0, 2, 0, None, 0, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == gdn.OK
    return out


# one CTA a unit, with one, three and eight warps' tiles to share; a cluster a unit; runs that cut units, several a CTA
CASES = {"unit": ([64] * 6, 8, 2, 1, 64), "rows": ([640] * 40, 12, 1, 3, 64), "wide": ([256] * 50, 8, 2, 1, 256),
         "cluster": ([3000], 8, 2, 1, 64), "runs": ([9000, 700, 100, 5000, 40, 40, 40], 8, 2, 1, 64)}


def case_of(name):
    lens, H, Hkv, n_q, dv = CASES[name]
    return Case(lens, H, Hkv, n_q, 64, dv, dtype="f16", seed=3, page=64)


@pytest.mark.parametrize("name", list(CASES))
def test_copies_land_before_their_warp_ends(X, name):
    """Whoever else waits for them: a CTA whose other warps gave up must not exit under copies into its memory."""
    c = case_of(name)
    want = c.run()
    assert X.look_at(1, -1, 0) == 0 and torch.equal(run(X, c), want)
    unseen = ctypes.c_int(-1)
    assert X.stages(ctypes.byref(unseen)) >= 4 and unseen.value == 0
    assert gdn.device_status() == gdn.OK


@pytest.mark.parametrize("name", list(CASES))
@pytest.mark.parametrize("warp", range(0, 16))
@pytest.mark.parametrize("lives", [0, 1, 7])
def test_a_wait_that_gives_up_ends_the_call(X, name, warp, lives):
    """Whichever warp's it is, the others agree on how to end: the call is over at once, the status word says so, no copy is
    left under way, and the next call is as ever."""
    c = case_of(name)
    want = c.run()
    torch.cuda.synchronize()
    assert gdn.device_status() == gdn.OK
    assert X.look_at(1, warp, lives) == 0
    run(X, c)
    lost, unseen = X.was_lost(), ctypes.c_int(-1)
    assert X.stages(ctypes.byref(unseen)) >= 0 and unseen.value == 0
    # (a warp without so many tiles has lost nothing; the first one has some)
    assert lost in (0, 1) and (lost or warp > 0 or lives > 0)
    assert gdn.device_status() == (gdn.ERR_TIMEOUT if lost else gdn.OK)
    assert torch.equal(c.run(), want)
