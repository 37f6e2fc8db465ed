"""GB300 (sm_103a) gated delta rule: Python binding of libgdn.so.

This module only marshals arguments: it checks torch tensors, takes their
device pointers and the current CUDA stream, and calls the C ABI declared in
``include/gdn.h``.  Every step of the computation runs in the library's CUDA
kernels; there is no CPU or PyTorch fallback.  If ``libgdn.so`` has not been
built (``python -m linear_attention_sequence_gated_gb300._build``) every
call raises.

    out, final_state = forward(q, k, v, g, beta, state)

q, k, v: (n_seqs, n_tokens, n_heads, head_dim) bf16 or fp32 CUDA tensors,
g, beta: (n_seqs, n_tokens, n_heads) fp32, state: (n_seqs, n_heads, head_dim,
head_dim) fp32 [value][key] or None (zeros).  out is fp32 and already carries
1/sqrt(head_dim).  ("marcsun13/ggml-gated-delta-net" model card, section
"Ops" and its shape table.)  q and k may carry fewer heads n_k (dividing
n_heads): value head i then reads key head i % n_k, the tiled mapping of the
model card's contract notes.

Beside it, for a hybrid's attention layers: ``flash_attn`` over dense keys and
values, and a paged 4-bit cache (``kv4_cache``, ``kv4_write``, ``kv4_read``,
``flash_attn_kv4``).  A decode step of a layer over that cache:

    lens += 1
    kv4_write(k, v, cache, page_table, lens)
    out = flash_attn_kv4(q, cache, page_table, lens)

and a paged cache of 16- or 32-bit rows (``paged_cache``, ``paged_write``,
``flash_attn_paged``) with rotary positions (``rotary_plan``, ``rotary``,
``rotary_write``).  Tables, slots and positions come from ``page_assign`` (the
tables serve the 4-bit cache too), and ``page_release`` takes pages back:

    lens += 1                                                      # once a step
    slots, positions, _ = page_assign(page_table, lens, free_pages, free_count, page_size)
    q = rotary_write(q, k, v, positions, plan, k_cache, v_cache, slots)     # each layer
    out = flash_attn_paged(q.unsqueeze(2), k_cache, v_cache, page_table, lens)
"""
from __future__ import annotations

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgdn.so")

OK = 0
ERR_ARG, ERR_HEADDIM, ERR_ALIGN, ERR_ALIAS, ERR_CUDA, ERR_TIMEOUT, ERR_WORKSPACE, ERR_NOMEM, \
    ERR_DTYPE, ERR_SHAPE, ERR_SCRATCH, ERR_PAGE = -1, -2, -3, -4, -5, -6, -7, -8, -9, -10, -11, -12
DTYPE_F32, DTYPE_BF16, DTYPE_F16 = 0, 1, 2
PATHS = {"auto": 0, "recurrent": 1, "chunked": 2}
OPT_L2NORM_QK = 0x100
OPT_OUT_BF16 = 0x200

# Every symbol include/gdn.h declares.
EXPORTS = ["gdn_forward", "gdn_forward_bf16", "gdn_forward_ex", "gdn_workspace_bytes",
           "gdn_select_path", "gdn_supports", "gdn_get_device_status", "gdn_status_string",
           "gdn_version", "gdn_flash_attn", "gdn_flash_attn_supports", "gdn_forward_noalloc",
           "gdn_selftest_wait_timeout", "gdn_kv4_supports", "gdn_kv4_cache_bytes", "gdn_kv4_write",
           "gdn_kv4_read", "gdn_flash_attn_kv4", "gdn_flash_attn_kv4_workspace_bytes",
           "gdn_page_assign", "gdn_page_release", "gdn_rotary_plan", "gdn_rotary", "gdn_paged_write",
           "gdn_rotary_write", "gdn_flash_attn_paged", "gdn_flash_attn_paged_workspace_bytes",
           "gdn_flash_attn_paged_supports"]
ROTARY_NEIGHBOURS, ROTARY_INVERSE = 1, 2

_lib = None


class GdnError(RuntimeError):
    def __init__(self, status: int, what: str = "gdn"):
        self.status = status
        super().__init__(f"{what} failed: {status_string(status)} ({status})")


def lib():
    """The loaded libgdn.so (ctypes), raising if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"libgdn.so not found at {LIB_PATH}; build it with "
                "`python -m linear_attention_sequence_gated_gb300._build` (no fallback exists)")
        L = ctypes.CDLL(LIB_PATH)
        vp, fp, i, sz = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        fwd = [vp, vp, vp, fp, fp, fp, fp, fp, i, i, i, i]
        L.gdn_forward.argtypes = fwd + [vp]
        L.gdn_forward_bf16.argtypes = fwd + [vp]
        L.gdn_forward_ex.argtypes = fwd[:11] + [i, i, i, i, vp, sz, vp]
        for f in (L.gdn_forward, L.gdn_forward_bf16, L.gdn_forward_ex):
            f.restype = i
        L.gdn_workspace_bytes.argtypes = [i, i, i, i, i, i]
        L.gdn_workspace_bytes.restype = sz
        L.gdn_select_path.argtypes = [i, i, i, i, i]
        L.gdn_select_path.restype = i
        L.gdn_supports.argtypes = [i]
        L.gdn_supports.restype = i
        L.gdn_get_device_status.argtypes = [vp]
        L.gdn_get_device_status.restype = i
        L.gdn_status_string.argtypes = [i]
        L.gdn_status_string.restype = ctypes.c_char_p
        L.gdn_version.restype = i
        L.gdn_flash_attn.argtypes = [vp, vp, vp, vp, fp] + [i] * 7 + [ctypes.c_float, i, vp]
        L.gdn_flash_attn.restype = i
        L.gdn_flash_attn_supports.argtypes = [i, i, i]
        L.gdn_flash_attn_supports.restype = i
        L.gdn_forward_noalloc.argtypes = fwd[:11] + [i, i, i, i, vp]
        L.gdn_forward_noalloc.restype = i
        L.gdn_selftest_wait_timeout.argtypes = [vp]
        L.gdn_selftest_wait_timeout.restype = i
        L.gdn_kv4_supports.argtypes = [i, i]
        L.gdn_kv4_supports.restype = i
        L.gdn_kv4_cache_bytes.argtypes = [i] * 5
        L.gdn_kv4_cache_bytes.restype = sz
        L.gdn_kv4_write.argtypes = [vp] * 7 + [i] * 9 + [vp]
        L.gdn_kv4_write.restype = i
        L.gdn_kv4_read.argtypes = [vp] * 6 + [i] * 9 + [vp]
        L.gdn_kv4_read.restype = i
        L.gdn_flash_attn_kv4.argtypes = [vp] * 6 + [i] * 9 + [ctypes.c_float, i, i, i, vp, sz, vp]
        L.gdn_flash_attn_kv4.restype = i
        L.gdn_flash_attn_kv4_workspace_bytes.argtypes = [i] * 8
        L.gdn_flash_attn_kv4_workspace_bytes.restype = sz
        L.gdn_page_assign.argtypes = [vp] * 8 + [i] * 6 + [vp]
        L.gdn_page_release.argtypes = [vp] * 5 + [i] * 4 + [vp]
        L.gdn_rotary_plan.argtypes = [vp, vp, i, vp]
        L.gdn_rotary.argtypes = [vp] * 7 + [i] * 8 + [vp]
        L.gdn_paged_write.argtypes = [vp] * 7 + [i] * 7 + [vp]
        L.gdn_rotary_write.argtypes = [vp] * 12 + [i] * 11 + [vp]
        L.gdn_flash_attn_paged.argtypes = [vp] * 9 + [i] * 9 + [ctypes.c_float, i, i, i, vp, sz, vp]
        for f in (L.gdn_page_assign, L.gdn_page_release, L.gdn_rotary_plan, L.gdn_rotary, L.gdn_paged_write,
                  L.gdn_rotary_write, L.gdn_flash_attn_paged):
            f.restype = i
        L.gdn_flash_attn_paged_workspace_bytes.argtypes = [i] * 9
        L.gdn_flash_attn_paged_workspace_bytes.restype = sz
        L.gdn_flash_attn_paged_supports.argtypes = [i, i, i]
        L.gdn_flash_attn_paged_supports.restype = i
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().gdn_status_string(int(status)).decode()


def supports(head_dim: int) -> int:
    """Bit mask: 1 = recurrent path, 2 = chunked path, 0 = unsupported."""
    return int(lib().gdn_supports(int(head_dim)))


def select_path(n_seqs: int, n_tokens: int, n_heads: int, head_dim: int,
                dtype: str = "bf16") -> str:
    """The path AUTO takes for these sizes: "recurrent" or "chunked"."""
    dt = DTYPE_BF16 if dtype in ("bf16", "bfloat16") else DTYPE_F32
    r = int(lib().gdn_select_path(int(n_seqs), int(n_tokens), int(n_heads), int(head_dim), dt))
    if r < 0:
        raise GdnError(r, "gdn_select_path")
    return {v: k for k, v in PATHS.items()}[r]


def workspace_bytes(n_seqs, n_tokens, n_heads, head_dim, dtype="bf16", path="auto") -> int:
    dt = DTYPE_BF16 if dtype in ("bf16", "bfloat16") else DTYPE_F32
    return int(lib().gdn_workspace_bytes(n_seqs, n_tokens, n_heads, head_dim, dt, PATHS[path]))


def device_status(stream=None) -> int:
    """Synchronise ``stream`` and return (and clear) the device status word."""
    return int(lib().gdn_get_device_status(_stream_handle(stream)))


def _stream_handle(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def forward(q, k, v, g, beta, state=None, *, out=None, state_out=None, path: str = "auto",
            workspace=None, stream=None, l2norm_qk: bool = False, out_dtype=None):
    """Run the gated delta rule over every token of every sequence.

    Returns (out, final_state).  ``state_out`` may be ``state`` itself for
    an in-place update.  ``workspace`` is an optional uint8 CUDA tensor of at
    least ``workspace_bytes(...)`` bytes; without it the library allocates
    stream-ordered scratch when the chosen path needs any.  ``l2norm_qk``
    divides q and k by their norm per (sequence, token, head) inside the op
    (the library's GDN_OPT_L2NORM_QK).  ``out_dtype`` torch.bfloat16 writes
    the output as bf16, each value the fp32 one rounded to nearest even
    (GDN_OPT_OUT_BF16); a given ``out`` must have that dtype.  The default is
    fp32, or the dtype of a given ``out``."""
    import torch
    L = lib()
    if q.dtype == torch.bfloat16:
        dt = DTYPE_BF16
    elif q.dtype == torch.float32:
        dt = DTYPE_F32
    else:
        raise TypeError(f"q/k/v must be bf16 or fp32, got {q.dtype}")
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be (n_seqs, n_tokens, heads, head_dim)")
    B, T, H, d = v.shape
    Hk = q.shape[2]
    if tuple(q.shape) != (B, T, Hk, d) or Hk < 1 or H % Hk != 0:
        raise ValueError(f"q: expected (n_seqs, n_tokens, n_k, head_dim) with n_k dividing "
                         f"{H}, got {tuple(q.shape)}")
    for name, t, shape, dtype in (("k", k, (B, T, Hk, d), q.dtype), ("v", v, (B, T, H, d), q.dtype),
                                  ("g", g, (B, T, H), torch.float32),
                                  ("beta", beta, (B, T, H), torch.float32)):
        if tuple(t.shape) != shape or t.dtype != dtype:
            raise ValueError(f"{name}: expected {shape} {dtype}, got {tuple(t.shape)} {t.dtype}")
    tensors = [q, k, v, g, beta]
    if state is not None:
        if tuple(state.shape) != (B, H, d, d) or state.dtype != torch.float32:
            raise ValueError("state must be (n_seqs, n_heads, head_dim, head_dim) fp32")
        tensors.append(state)
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.float32
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"out_dtype must be float32 or bfloat16, got {out_dtype}")
    if out is None:
        out = torch.empty((B, T, H, d), dtype=out_dtype, device=q.device)
    if state_out is None:
        state_out = torch.empty((B, H, d, d), dtype=torch.float32, device=q.device)
    tensors += [out, state_out]
    for t in tensors:
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("all tensors must be contiguous CUDA tensors")
        if t.device != q.device:
            raise ValueError("all tensors must be on one CUDA device")
    if tuple(out.shape) != (B, T, H, d) or out.dtype != out_dtype:
        raise ValueError(f"out must be (n_seqs, n_tokens, n_heads, head_dim) {out_dtype}")
    if tuple(state_out.shape) != (B, H, d, d) or state_out.dtype != torch.float32:
        raise ValueError("state_out must be (n_seqs, n_heads, head_dim, head_dim) fp32")
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        ws_ptr, ws_bytes = _ptr(workspace), workspace.numel() * workspace.element_size()
    with torch.cuda.device(q.device):
        rc = L.gdn_forward_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state),
                              _ptr(out), _ptr(state_out), B, T, H, Hk, d, dt,
                              PATHS[path] | (OPT_L2NORM_QK if l2norm_qk else 0)
                              | (OPT_OUT_BF16 if out_dtype == torch.bfloat16 else 0),
                              ws_ptr, ws_bytes, _stream_handle(stream))
    if rc != OK:
        raise GdnError(rc, "gdn_forward_ex")
    return out, state_out


def flash_attn_supports(n_q: int, head_dim_k: int, head_dim_v: int) -> bool:
    """Whether ``flash_attn`` serves this shape (fewer than 20 queries; key and
    value head dims each 64, 128 or 256, equal or not)."""
    return bool(lib().gdn_flash_attn_supports(int(n_q), int(head_dim_k), int(head_dim_v)))


def flash_attn(q, k, v, mask=None, scale=None, *, out=None, stream=None):
    """Decode attention: out[b, i, h] = softmax_j(scale q[b,h,i] . k[b,hk,j] +
    mask[b,0,i,j]) v[b,hk,j], hk = h // (n_heads / n_heads_kv).

    q: (n_seqs, n_heads, n_q, dk); k: (n_seqs, n_heads_kv, n_kv, dk); v:
    (n_seqs, n_heads_kv, n_kv, dv), all of one dtype (fp32, bf16 or fp16);
    mask: (n_seqs, 1, n_q, n_kv) of the same dtype, additive, or None; scale
    defaults to 1/sqrt(dk).  Returns out (n_seqs, n_q, n_heads, dv) fp32.  ("marcsun13/ggml-gated-delta-net" model
    card, section "flash_attn".)"""
    import math
    import torch
    L = lib()
    dts = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16}
    if q.dtype not in dts:
        raise TypeError(f"q/k/v must be fp32, bf16 or fp16, got {q.dtype}")
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be 4-D")
    B, H, n_q, dk = q.shape
    Hkv, n_kv = k.shape[1], k.shape[2]
    dv = v.shape[3]
    if tuple(k.shape) != (B, Hkv, n_kv, dk) or tuple(v.shape) != (B, Hkv, n_kv, dv):
        raise ValueError(f"k, v: expected (n_seqs, n_heads_kv, n_kv, dk / dv), got {tuple(k.shape)}, "
                         f"{tuple(v.shape)}")
    tensors = [q, k, v]
    if mask is not None:
        if tuple(mask.shape) != (B, 1, n_q, n_kv):
            raise ValueError(f"mask: expected {(B, 1, n_q, n_kv)}, got {tuple(mask.shape)}")
        tensors.append(mask)
    for t in tensors:
        if t.dtype != q.dtype:
            raise TypeError("q, k, v and mask must share one dtype")
    if out is None:
        out = torch.empty((B, n_q, H, dv), dtype=torch.float32, device=q.device)
    tensors.append(out)
    for t in tensors:
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("all tensors must be contiguous CUDA tensors")
        if t.device != q.device:
            raise ValueError("all tensors must be on one CUDA device")
    if tuple(out.shape) != (B, n_q, H, dv) or out.dtype != torch.float32:
        raise ValueError("out must be (n_seqs, n_q, n_heads, dv) fp32")
    if scale is None:
        scale = 1.0 / math.sqrt(dk)
    with torch.cuda.device(q.device):
        rc = L.gdn_flash_attn(_ptr(q), _ptr(k), _ptr(v), _ptr(mask), _ptr(out), B, H, Hkv, n_q,
                              n_kv, dk, dv, float(scale), dts[q.dtype], _stream_handle(stream))
    if rc != OK:
        raise GdnError(rc, "gdn_flash_attn")
    return out


# ------------------------------------------------------------------ 4-bit cache
#
# A decode step makes these calls once a layer, so their host side is kept short:
# no imports, context managers or Stream objects where the current device and
# stream serve.

_torch = None
_KV4_DTYPES = {}


def _kv4_torch():
    """The torch module, and the library's codes of its dtypes filled in."""
    global _torch
    if _torch is None:
        import torch
        _KV4_DTYPES.update({torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16})
        _torch = torch
    return _torch


def _kv4_dtype(dtype, what):
    code = _KV4_DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"{what} must be fp32, bf16 or fp16, got {dtype}")
    return code


def _kv4_check(torch, cache, page_table, seq_lens, B, Hkv, dk, dv, lens=None):
    """Shapes, types and devices of a cache and what goes with it; its device's
    index, pages, tokens of a page and pages of a sequence's table."""
    shape, width, int32 = cache.shape, 9 * (dk + dv), torch.int32
    if len(shape) != 4 or shape[1] != Hkv or shape[3] != width or cache.dtype != torch.uint8:
        raise ValueError(f"cache: expected (n_pages, {Hkv}, page_size / 16, {width}) uint8, got "
                         f"{tuple(shape)} {cache.dtype}")
    pages = page_table.shape
    if len(pages) != 2 or pages[0] != B or page_table.dtype != int32:
        raise ValueError(f"page_table: expected ({B}, max_pages) int32, got {tuple(pages)} "
                         f"{page_table.dtype}")
    dev = cache.get_device()
    for t in (seq_lens,) if lens is None else (seq_lens, lens):
        if t.shape != (B,) or t.dtype != int32:
            raise ValueError(f"lengths: expected ({B},) int32, got {tuple(t.shape)} {t.dtype}")
        if t.get_device() != dev or not t.is_contiguous():
            raise ValueError("lengths must be contiguous and on the cache's device")
    if dev < 0 or page_table.get_device() != dev or not cache.is_contiguous() or not page_table.is_contiguous():
        raise ValueError("cache and page_table must be contiguous CUDA tensors on one device")
    return dev, shape[0], shape[2] * 16, pages[1]


def _kv4_call(torch, dev, stream, call):
    """call(handle of the stream to run on), with ``dev`` current, and ``stream``
    too if one is given, so that what the call allocates belongs to its stream."""
    if stream is not None:
        if stream.device.index != dev:
            raise ValueError("stream must be on the tensors' device")
        with torch.cuda.stream(stream):
            return call(stream.cuda_stream)
    if dev == torch._C._cuda_getDevice():
        return call(torch._C._cuda_getCurrentRawStream(dev))
    with torch.cuda.device(dev):
        return call(torch._C._cuda_getCurrentRawStream(dev))


def kv4_supports(head_dim_k: int, head_dim_v: int) -> bool:
    """Whether the 4-bit cache serves these widths (each 64, 128 or 256)."""
    return bool(lib().gdn_kv4_supports(int(head_dim_k), int(head_dim_v)))


def kv4_cache(n_pages: int, n_heads_kv: int, page_size: int, head_dim_k: int, head_dim_v=None, *,
              device="cuda"):
    """An empty 4-bit cache: (n_pages, n_heads_kv, page_size / 16, 9 (dk + dv))
    uint8, for keys of ``head_dim_k`` and values of ``head_dim_v`` (the same
    where it is not given).  page_size is a multiple of 16."""
    torch = _kv4_torch()
    dv = head_dim_k if head_dim_v is None else head_dim_v
    if not kv4_supports(head_dim_k, dv):
        raise GdnError(ERR_HEADDIM, "kv4_cache")
    if page_size < 16 or page_size % 16 != 0:
        raise GdnError(ERR_SHAPE, "kv4_cache")
    return torch.zeros((n_pages, n_heads_kv, page_size // 16, 9 * (head_dim_k + dv)), dtype=torch.uint8,
                       device=device)


def kv4_write(k, v, cache, page_table, seq_lens, new_lens=None, *, stream=None):
    """Quantise new rows into a 4-bit cache and return the cache.

    k: (n_seqs, n_heads_kv, n_new, dk), v: (n_seqs, n_heads_kv, n_new, dv), fp32,
    bf16 or fp16; any strides with contiguous, 16-byte aligned rows (a transposed
    view of token-major projections needs no copy).  page_table: (n_seqs,
    max_pages) int32; seq_lens: (n_seqs,) int32, lengths that count the new
    tokens: token i of sequence b goes to position seq_lens[b] - n + i, n =
    new_lens[b] or n_new.  Tokens from n on and at negative positions are not
    written.  A page outside the cache shows as ERR_PAGE in device_status().
    The format and the rest of the contract are with gdn_kv4_write in
    include/gdn.h."""
    L, torch = lib(), _kv4_torch()
    dt = _kv4_dtype(k.dtype, "k/v")
    kn, vn = k.shape, v.shape
    if len(kn) != 4 or len(vn) != 4 or vn[:3] != kn[:3] or v.dtype != k.dtype:
        raise ValueError("k, v: expected (n_seqs, n_heads_kv, n_new, dk / dv) of one dtype, got "
                         f"{tuple(kn)} {k.dtype}, {tuple(vn)} {v.dtype}")
    B, Hkv, T, dk = kn
    dv = vn[3]
    dev, n_pages, page, max_pages = _kv4_check(torch, cache, page_table, seq_lens, B, Hkv, dk, dv, new_lens)
    ks, vs = k.stride(), v.stride()
    if k.get_device() != dev or v.get_device() != dev:
        raise ValueError("all tensors must be on one CUDA device")
    if (ks[3] != 1 or vs[3] != 1) and k.numel():
        raise ValueError("rows of k and v must be contiguous")
    strides = None if k.is_contiguous() and v.is_contiguous() else \
        (ctypes.c_longlong * 6)(ks[0], ks[1], ks[2], vs[0], vs[1], vs[2])

    def call(handle):
        return L.gdn_kv4_write(k.data_ptr(), v.data_ptr(), strides, cache.data_ptr(), page_table.data_ptr(),
                               seq_lens.data_ptr(), None if new_lens is None else new_lens.data_ptr(), B, T,
                               Hkv, dk, dv, n_pages, page, max_pages, dt, handle)

    rc = _kv4_call(torch, dev, stream, call)
    if rc != OK:
        raise GdnError(rc, "gdn_kv4_write")
    return cache


def kv4_read(cache, page_table, seq_lens, n_tokens: int, head_dim_k: int, head_dim_v=None, *, lens=None,
             dtype=None, k_out=None, v_out=None, stream=None):
    """The last rows of each sequence in a 4-bit cache, dense: (k, v) of shapes
    (n_seqs, n_heads_kv, n_tokens, dk) and (..., dv), as flash_attn takes them.

    Row i of sequence b is what is kept at position seq_lens[b] - n + i, n =
    lens[b] or n_tokens (what a kv4_write of the same lengths wrote); rows from n
    on and at negative positions are zeros.  With lens = seq_lens row i is
    position i.  ``dtype``: fp32, bf16 (default) or fp16; every value is exact
    in each."""
    L, torch = lib(), _kv4_torch()
    dk, dv = int(head_dim_k), int(head_dim_k if head_dim_v is None else head_dim_v)
    if dtype is None:
        dtype = k_out.dtype if k_out is not None else torch.bfloat16
    dt = _kv4_dtype(dtype, "dtype")
    if cache.dim() != 4 or page_table.dim() != 2:
        raise ValueError("cache must be 4-D and page_table 2-D")
    B, Hkv = page_table.shape[0], cache.shape[1]
    dev, n_pages, page, max_pages = _kv4_check(torch, cache, page_table, seq_lens, B, Hkv, dk, dv, lens)
    for name, t, d in (("k_out", k_out, dk), ("v_out", v_out, dv)):
        if t is not None and (tuple(t.shape) != (B, Hkv, n_tokens, d) or t.dtype != dtype
                              or not t.is_contiguous() or t.get_device() != dev):
            raise ValueError(f"{name} must be contiguous {(B, Hkv, n_tokens, d)} {dtype} on the cache's device")

    def call(handle):
        k = torch.empty((B, Hkv, n_tokens, dk), dtype=dtype, device=cache.device) if k_out is None else k_out
        v = torch.empty((B, Hkv, n_tokens, dv), dtype=dtype, device=cache.device) if v_out is None else v_out
        rc = L.gdn_kv4_read(cache.data_ptr(), page_table.data_ptr(), seq_lens.data_ptr(),
                            None if lens is None else lens.data_ptr(), k.data_ptr(), v.data_ptr(), B, n_tokens,
                            Hkv, dk, dv, n_pages, page, max_pages, dt, handle)
        if rc != OK:
            raise GdnError(rc, "gdn_kv4_read")
        return k, v

    return _kv4_call(torch, dev, stream, call)


def flash_attn_kv4_workspace_bytes(n_seqs, n_heads, n_heads_kv, n_q, head_dim_k, head_dim_v, page_size,
                                   max_pages) -> int:
    """Bytes that ``flash_attn_kv4`` needs as its ``workspace`` (0: none)."""
    return int(lib().gdn_flash_attn_kv4_workspace_bytes(n_seqs, n_heads, n_heads_kv, n_q, head_dim_k,
                                                        head_dim_v, page_size, max_pages))


def flash_attn_kv4(q, cache, page_table, seq_lens, head_dim_v=None, mask=None, scale=None, *,
                   causal: bool = False, out=None, out_dtype=None, workspace=None, stream=None):
    """Decode attention over a 4-bit cache: out[b, i, h] = softmax_j(scale
    q[b,h,i] . k[b,hk,j] + mask[b,0,i,j]) v[b,hk,j] over the seq_lens[b] tokens of
    each sequence (with ``causal``, j <= seq_lens[b] - n_q + i), hk = h //
    (n_heads / n_heads_kv).

    q: (n_seqs, n_heads, n_q, dk) fp32, bf16 or fp16; cache, page_table,
    seq_lens as for kv4_write; head_dim_v: the values' width (default dk); mask:
    (n_seqs, 1, n_q, max_pages * page_size) of q's dtype, additive, or None; scale
    defaults to 1/sqrt(dk).  Returns out (n_seqs, n_q, n_heads, dv) of
    ``out_dtype`` (fp32 by default, or a given out's dtype).  Rows that see no
    token are zeros.  ``workspace``: an optional uint8 CUDA tensor of
    flash_attn_kv4_workspace_bytes(...) bytes for one call at a time; without it
    the library allocates in stream order."""
    L, torch = lib(), _kv4_torch()
    dt = _kv4_dtype(q.dtype, "q")
    if q.dim() != 4 or cache.dim() != 4:
        raise ValueError("q and cache must be 4-D")
    B, H, n_q, dk = q.shape
    dv = int(dk if head_dim_v is None else head_dim_v)
    Hkv = cache.shape[1]
    dev, n_pages, page, max_pages = _kv4_check(torch, cache, page_table, seq_lens, B, Hkv, dk, dv)
    if mask is not None and (tuple(mask.shape) != (B, 1, n_q, max_pages * page) or mask.dtype != q.dtype):
        raise ValueError(f"mask: expected {(B, 1, n_q, max_pages * page)} {q.dtype}, got "
                         f"{tuple(mask.shape)} {mask.dtype}")
    for t in (q, mask, workspace):
        if t is not None and (t.get_device() != dev or not t.is_contiguous()):
            raise ValueError("all tensors must be contiguous CUDA tensors on one device")
    if out is not None:
        if out_dtype is None:
            out_dtype = out.dtype
        if tuple(out.shape) != (B, n_q, H, dv) or out.dtype != out_dtype or not out.is_contiguous() \
                or out.get_device() != dev:
            raise ValueError(f"out must be contiguous {(B, n_q, H, dv)} {out_dtype} on the cache's device")
    elif out_dtype is None:
        out_dtype = torch.float32
    odt = _kv4_dtype(out_dtype, "out_dtype")
    if scale is None:
        scale = dk ** -0.5

    def call(handle):
        o = torch.empty((B, n_q, H, dv), dtype=out_dtype, device=cache.device) if out is None else out
        rc = L.gdn_flash_attn_kv4(
            q.data_ptr(), cache.data_ptr(), page_table.data_ptr(), seq_lens.data_ptr(),
            None if mask is None else mask.data_ptr(), o.data_ptr(), B, H, Hkv, n_q, dk, dv, n_pages,
            page, max_pages, scale, 1 if causal else 0, dt, odt,
            None if workspace is None else workspace.data_ptr(),
            0 if workspace is None else workspace.numel() * workspace.element_size(), handle)
        if rc != OK:
            raise GdnError(rc, "gdn_flash_attn_kv4")
        return o

    return _kv4_call(torch, dev, stream, call)


# ------------------------------------------------------- pages, rotary positions, 16- and 32-bit cache
#
# Each call first looks whether its arguments are as expected, in as few steps as it takes; what is
# wrong with the others is found out afterwards (_refuse), and strides go along only where a tensor is not dense.
# Where another device is current, or a stream is given, the call makes them current and starts again (_there).


def _refuse(checks):
    """Raise for the first (name, tensor, shape, dtype, device index) that is not so; None in a shape: any size."""
    for name, t, shape, dtype, dev in checks:
        if t is None:
            continue
        if len(t.shape) != len(shape) or any(w is not None and w != n for w, n in zip(shape, t.shape)) or t.dtype != dtype:
            want = "(" + ", ".join("any" if w is None else str(w) for w in shape) + ")"
            raise ValueError(f"{name}: expected {want} {dtype}, got {tuple(t.shape)} {t.dtype}")
        if dev < 0 or t.get_device() != dev:
            raise ValueError(f"{name}: all tensors must be on one CUDA device")
        if dtype == _torch.int32 and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if t.numel() and t.stride(-1) != 1:
            raise ValueError(f"rows of {name} must be contiguous")
    raise ValueError("arguments do not fit together")


def _there(dev, stream, call, *args, **kw):
    """call(*args, **kw) with ``dev`` current, and ``stream`` too if one is given, so that what the call
    allocates belongs to its stream."""
    if stream is None:
        with _torch.cuda.device(dev):
            return call(*args, **kw)
    if stream.device.index != dev:
        raise ValueError("stream must be on the tensors' device")
    with _torch.cuda.stream(stream):
        return call(*args, **kw)


def _strides(*xs):
    """Host array of the strides of every dimension but the last."""
    v = [s for x in xs for s in x.stride()[:-1]]
    return (ctypes.c_longlong * len(v))(*v)


def page_assign(page_table, seq_lens, free_pages, free_count, page_size: int, n_new=None, new_lens=None, *,
                n_tokens=None, slots=None, positions=None, offsets=None, stream=None):
    """Pages, slots and positions for a step's new tokens; returns (slots, positions, offsets).

    page_table (n_seqs, max_pages), seq_lens (n_seqs), free_pages (n_pages),
    free_count (1), new_lens (n_seqs, at most n_new each) or None (n_new each): int32.
    n_new defaults to 1, or to n_tokens where that and new_lens are given (as far as n_seqs times
    it is below 2^31).  seq_lens count the new tokens.  Pages that they are the first to need leave the stack
    free_pages[:free_count] from its end and enter the table; free_count and the
    table are updated in place.  Without ``n_tokens`` slots and positions are
    (n_seqs, n_new), -1 and 0 where there is no token, and offsets is None; with it
    they are packed, (n_tokens,), sequence b's from offsets[b] on, offsets
    (n_seqs + 1).  A stack that runs out, a new_lens entry above n_new, and whatever else only the device can
    see, shows as ERR_PAGE in device_status().  The rest of the contract is with
    gdn_page_assign in include/gdn.h."""
    L, torch = _lib or lib(), _torch or _kv4_torch()
    i32, dev, table, lens, pool = torch.int32, page_table.get_device(), page_table.shape, seq_lens.shape, free_pages.shape
    B = table[0] if table else 0
    packed = n_tokens is not None
    if not (dev >= 0 and len(table) == 2 and page_table.dtype is i32 and page_table.is_contiguous()
            and len(lens) == 1 and lens[0] == B and seq_lens.dtype is i32 and seq_lens.get_device() == dev
            and seq_lens.is_contiguous()
            and len(pool) == 1 and free_pages.dtype is i32 and free_pages.get_device() == dev
            and free_pages.is_contiguous()
            and free_count.shape == (1,) and free_count.dtype is i32 and free_count.get_device() == dev
            and (new_lens is None or (new_lens.shape == lens and new_lens.dtype is i32
                                      and new_lens.get_device() == dev and new_lens.is_contiguous()))):
        _refuse((("page_table", page_table, (None, None), i32, dev), ("seq_lens", seq_lens, (B,), i32, dev),
                 ("free_pages", free_pages, (None,), i32, dev), ("free_count", free_count, (1,), i32, dev),
                 ("new_lens", new_lens, (B,), i32, dev)))
    if n_new is None:
        n_new = 1 if not packed or new_lens is None else min(n_tokens, 0x7fffffff // max(B, 1))
    if stream is not None or torch._C._cuda_getDevice() != dev:
        return _there(dev, stream, page_assign, page_table, seq_lens, free_pages, free_count, page_size, n_new, new_lens,
                      n_tokens=n_tokens, slots=slots, positions=positions, offsets=offsets)
    shape = (n_tokens,) if packed else (B, n_new)
    for name, t, want in (("slots", slots, shape), ("positions", positions, shape), ("offsets", offsets, (B + 1,))):
        if t is not None and not (t.shape == want and t.dtype is i32 and t.get_device() == dev and t.is_contiguous()):
            _refuse(((name, t, want, i32, dev),))
    if offsets is not None and not packed:
        raise ValueError("offsets go with n_tokens")
    if slots is None:
        slots = torch.empty(shape, dtype=i32, device=page_table.device)
    if positions is None:
        positions = torch.empty(shape, dtype=i32, device=page_table.device)
    if packed and offsets is None:
        offsets = torch.empty((B + 1,), dtype=i32, device=page_table.device)
    rc = L.gdn_page_assign(page_table.data_ptr(), seq_lens.data_ptr(), None if new_lens is None else new_lens.data_ptr(),
                           free_pages.data_ptr(), free_count.data_ptr(), slots.data_ptr(), positions.data_ptr(),
                           offsets.data_ptr() if packed else None, B, n_new, n_tokens if packed else 0, page_size,
                           table[1], pool[0], torch._C._cuda_getCurrentRawStream(dev))
    if rc != OK:
        raise GdnError(rc, "gdn_page_assign")
    return slots, positions, offsets


def page_release(page_table, from_lens, free_pages, free_count, page_size: int, to_lens=None, *, stream=None):
    """Give back the pages of sequences that shrink from ``from_lens`` to ``to_lens`` tokens (None: to none).

    Arguments as for page_assign; free_pages and free_count are updated in place.
    A step called off (to_lens: the lengths before it) leaves the stack as it was."""
    L, torch = _lib or lib(), _torch or _kv4_torch()
    i32, dev, table, lens, pool = torch.int32, page_table.get_device(), page_table.shape, from_lens.shape, free_pages.shape
    B = table[0] if table else 0
    if not (dev >= 0 and len(table) == 2 and page_table.dtype is i32 and page_table.is_contiguous()
            and len(lens) == 1 and lens[0] == B and from_lens.dtype is i32 and from_lens.get_device() == dev
            and from_lens.is_contiguous()
            and len(pool) == 1 and free_pages.dtype is i32 and free_pages.get_device() == dev
            and free_pages.is_contiguous()
            and free_count.shape == (1,) and free_count.dtype is i32 and free_count.get_device() == dev
            and (to_lens is None or (to_lens.shape == lens and to_lens.dtype is i32
                                     and to_lens.get_device() == dev and to_lens.is_contiguous()))):
        _refuse((("page_table", page_table, (None, None), i32, dev), ("from_lens", from_lens, (B,), i32, dev),
                 ("free_pages", free_pages, (None,), i32, dev), ("free_count", free_count, (1,), i32, dev),
                 ("to_lens", to_lens, (B,), i32, dev)))
    if stream is not None or torch._C._cuda_getDevice() != dev:
        return _there(dev, stream, page_release, page_table, from_lens, free_pages, free_count, page_size, to_lens)
    rc = L.gdn_page_release(page_table.data_ptr(), from_lens.data_ptr(), None if to_lens is None else to_lens.data_ptr(),
                            free_pages.data_ptr(), free_count.data_ptr(), B, page_size, table[1], pool[0],
                            torch._C._cuda_getCurrentRawStream(dev))
    if rc != OK:
        raise GdnError(rc, "gdn_page_release")


class RotaryPlan:
    """Frequencies of rotary positions on a device, made by rotary_plan."""

    def __init__(self, data, rot_dim, n_axes, neighbours):
        self.data, self.rot_dim, self.n_axes, self.neighbours = data, rot_dim, n_axes, neighbours
        # what every call hands on
        self._ptr, self._dev, self._flags = data.data_ptr(), data.get_device(), ROTARY_NEIGHBOURS if neighbours else 0


def rotary_plan(rot_dim: int, base: float = 10000.0, *, freqs=None, sections=None, dealt: bool = False,
                neighbours: bool = False, device="cuda"):
    """A plan for ``rotary`` and ``rotary_write``: pair j of a row's first ``rot_dim`` elements turns by its
    axis's position times base ** (-2 j / rot_dim), or times freqs[j] (radians a position) where given.

    sections: how many frequencies belong to each axis (their sum is rot_dim / 2;
    default one axis), one axis after another, or with ``dealt`` dealt out in turn
    (0, 1, 2, 0, 1, 2, ...) while an axis has any left.  Pairs are elements j and j + rot_dim / 2, or with
    ``neighbours`` 2 j and 2 j + 1."""
    L, torch = lib(), _kv4_torch()
    n = rot_dim // 2
    if rot_dim < 0 or rot_dim % 16 != 0:
        raise GdnError(ERR_HEADDIM, "rotary_plan")
    f = [float(base) ** (-2.0 * j / rot_dim) for j in range(n)] if freqs is None else [float(x) for x in freqs]
    left = [n] if sections is None else [int(x) for x in sections]
    if len(f) != n or not left or min(left) < 0 or sum(left) != n:
        raise ValueError(f"expected {n} frequencies, and sections of as many in all")
    n_axes, axes = len(left), []
    if dealt:
        while len(axes) < n:
            for a in range(n_axes):
                if left[a] > 0:
                    axes.append(a)
                    left[a] -= 1
    else:
        axes = [a for a in range(n_axes) for _ in range(left[a])]
    host = torch.zeros((n, 2), dtype=torch.int64)
    rc = L.gdn_rotary_plan((ctypes.c_double * n)(*f), (ctypes.c_int * n)(*axes), n, host.data_ptr())
    if rc != OK:
        raise GdnError(rc, "gdn_rotary_plan")
    return RotaryPlan(host.to(device), rot_dim, n_axes, bool(neighbours))


_rotary_node = None


def _rotary_function():
    """rotary as a node of autograd, whose backward pass is rotary again (so it has a gradient too)."""
    global _rotary_node
    if _rotary_node is not None:
        return _rotary_node

    def rows(g):
        """g, or a dense copy where its rows are not as rotary takes them (the gradient of a sum is one element)."""
        ok = g.stride(2) == 1 and g.data_ptr() % 16 == 0 and not any(
            g.stride(i) * g.element_size() % 16 for i in (0, 1) if g.shape[i] > 1)
        return g if ok else g.clone(memory_format=_torch.contiguous_format)

    class Rotary(_torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, positions, plan, inverse):
            ctx.set_materialize_grads(False)
            ctx.save_for_backward(positions)
            ctx.plan, ctx.inverse = plan, inverse
            return rotary(q, k, positions, plan, inverse=inverse)

        @staticmethod
        def backward(ctx, dq, dk):
            positions, = ctx.saved_tensors
            grads = [rows(g) if g is not None and need else None for g, need in zip((dq, dk), ctx.needs_input_grad)]
            some = [g for g in grads if g is not None]
            if some:
                turned = list(rotary(some[0], some[1] if len(some) > 1 else None, positions, ctx.plan,
                                     inverse=not ctx.inverse))
                grads = [None if g is None else turned.pop(0) for g in grads]
            return (*grads, None, None, None)

    _rotary_node = Rotary
    return Rotary


def rotary(q, k, positions, plan, *, inverse: bool = False, q_out=None, k_out=None, stream=None):
    """Turn pairs of elements of q (n_tokens, n_heads, head_dim) and k (n_tokens, n_heads_kv, head_dim, or
    None) by their tokens' positions; returns (q_out, k_out).

    positions: (n_tokens,) int32, or (n_axes, n_tokens) for a plan of several
    axes.  fp32, bf16 or fp16; any strides with contiguous, 16-byte aligned rows.
    q_out and k_out may be q and k themselves (default: new dense tensors).
    ``inverse`` turns back, which is also the gradient: rotary(dq_out, dk_out,
    positions, plan, inverse=True) is (dq, dk).  Where q or k requires a gradient, autograd gets just that from the
    results; given outputs are plain memory to it, as with every other call here."""
    L, torch = _lib or lib(), _torch or _kv4_torch()
    dtype, dev, qs, i32, axes, ps = q.dtype, q.get_device(), q.shape, torch.int32, plan.n_axes, positions.shape
    dt = _KV4_DTYPES.get(dtype)
    if dt is None or len(qs) != 3:
        _kv4_dtype(dtype, "q")
        raise ValueError(f"q: expected (n_tokens, n_heads, head_dim), got {tuple(qs)}")
    T, H, d = qs
    ks = (T, 0, d) if k is None else k.shape
    if not (dev >= 0 and plan._dev == dev
            and (k is None or (len(ks) == 3 and ks[0] == T and ks[2] == d and k.dtype is dtype and k.get_device() == dev))
            and positions.dtype is i32 and positions.get_device() == dev and positions.is_contiguous()
            and (ps == (axes, T) or (axes == 1 and ps == (T,)))):
        _refuse((("q", q, (None, None, None), dtype, dev), ("k", k, (T, None, d), dtype, dev),
                 ("plan", plan.data, (plan.rot_dim // 2, 2), torch.int64, dev),
                 ("positions", positions, (T,) if len(ps) == 1 and axes == 1 else (axes, T), i32, dev)))
    if stream is not None or torch._C._cuda_getDevice() != dev:
        return _there(dev, stream, rotary, q, k, positions, plan, inverse=inverse, q_out=q_out, k_out=k_out)
    if (q.requires_grad or (k is not None and k.requires_grad)) and q_out is None and k_out is None \
            and torch.is_grad_enabled():
        return _rotary_function().apply(q, k, positions, plan, inverse)
    dense = q.is_contiguous() and (k is None or k.is_contiguous())
    if q_out is None:
        q_out = torch.empty_like(q) if dense else torch.empty(qs, dtype=dtype, device=q.device)
    elif not (q_out.shape == qs and q_out.dtype is dtype and q_out.get_device() == dev):
        _refuse((("q_out", q_out, tuple(qs), dtype, dev),))
    elif not q_out.is_contiguous():
        dense = False
    if k is None:
        if k_out is not None:
            raise ValueError("k_out goes with k")
    elif k_out is None:
        k_out = torch.empty_like(k) if dense else torch.empty(ks, dtype=dtype, device=q.device)
    elif not (k_out.shape == ks and k_out.dtype is dtype and k_out.get_device() == dev):
        _refuse((("k_out", k_out, tuple(ks), dtype, dev),))
    elif not k_out.is_contiguous():
        dense = False
    strides = None
    if not dense:
        every = (q, q_out, q, q_out) if k is None else (q, q_out, k, k_out)
        if any(t.stride(2) != 1 and t.numel() for t in every):
            raise ValueError("rows must be contiguous")
        strides = _strides(*every)
    rc = L.gdn_rotary(q.data_ptr(), q_out.data_ptr(), None if k is None else k.data_ptr(),
                      None if k is None else k_out.data_ptr(), strides, positions.data_ptr(), plan._ptr, T, H, ks[1], d,
                      plan.rot_dim, axes, plan._flags | ROTARY_INVERSE if inverse else plan._flags, dt,
                      torch._C._cuda_getCurrentRawStream(dev))
    if rc != OK:
        raise GdnError(rc, "gdn_rotary")
    return q_out, k_out


def paged_cache(n_pages: int, n_heads_kv: int, page_size: int, head_dim_k: int, head_dim_v=None, *, dtype=None,
                device="cuda"):
    """An empty cache of 16- or 32-bit rows: (k_cache, v_cache) of shapes (n_pages, n_heads_kv, page_size, dk) and
    (..., dv), bf16 where no dtype is given.  The calls below take any strides that nest (pages may be
    token-major: a transposed view of (n_pages, page_size, n_heads_kv, dk)).  Rows of any multiple of 16 elements up to
    256 can be written; flash_attn_paged reads widths of 64, 128 and 256 and pages of a multiple of 16 tokens."""
    torch = _kv4_torch()
    dtype = torch.bfloat16 if dtype is None else dtype
    _kv4_dtype(dtype, "dtype")
    dv = head_dim_k if head_dim_v is None else head_dim_v
    return tuple(torch.empty((n_pages, n_heads_kv, page_size, d), dtype=dtype, device=device) for d in (head_dim_k, dv))


def paged_write(k, v, k_cache, v_cache, slots, *, stream=None):
    """Copy rows k, v (n_tokens, n_heads_kv, dk / dv) to their slots; returns (k_cache, v_cache).

    slots: (n_tokens,) int32 as page_assign gives them (a padded batch's flattened),
    negative: not written; they must differ."""
    _write_rows(None, k, v, None, None, k_cache, v_cache, slots, None, stream)
    return k_cache, v_cache


def rotary_write(q, k, v, positions, plan, k_cache, v_cache, slots, *, q_out=None, stream=None):
    """rotary of q and k and paged_write of the turned k and of v, in one launch; returns q_out (default: a new dense
    tensor; may be q itself).  Arguments as for rotary and paged_write."""
    if q is None or plan is None:
        raise TypeError("rotary_write takes queries and a plan (paged_write: neither)")
    return _write_rows(q, k, v, positions, plan, k_cache, v_cache, slots, q_out, stream)


def _write_rows(q, k, v, positions, plan, k_cache, v_cache, slots, q_out, stream):
    L, torch = _lib or lib(), _torch or _kv4_torch()
    dtype, dev, ks, vs, cs, ws, i32 = k.dtype, k.get_device(), k.shape, v.shape, k_cache.shape, v_cache.shape, torch.int32
    dt = _KV4_DTYPES.get(dtype)
    if dt is None:
        _kv4_dtype(dtype, "k/v")
    if not (dev >= 0 and len(ks) == 3 and len(vs) == 3 and len(cs) == 4 and len(ws) == 4
            and vs[0] == ks[0] and cs[0] == ws[0] and cs[2] == ws[2] and ks[1] == vs[1] == cs[1] == ws[1]
            and cs[3] == ks[2] and ws[3] == vs[2]
            and v.dtype is dtype and k_cache.dtype is dtype and v_cache.dtype is dtype
            and v.get_device() == dev and k_cache.get_device() == dev and v_cache.get_device() == dev
            and slots.shape == (ks[0],) and slots.dtype is i32 and slots.get_device() == dev and slots.is_contiguous()):
        H = ks[1] if len(ks) == 3 else None
        _refuse((("k", k, (None, None, None), dtype, dev), ("v", v, (ks[0], H, None), dtype, dev),
                 ("k_cache", k_cache, (None, H, None, ks[-1]), dtype, dev),
                 ("v_cache", v_cache, tuple(cs[:1]) + (H,) + tuple(cs[2:3]) + (vs[-1],), dtype, dev),
                 ("slots", slots, (ks[0],), i32, dev)))
    if stream is not None or torch._C._cuda_getDevice() != dev:
        return _there(dev, stream, _write_rows, q, k, v, positions, plan, k_cache, v_cache, slots, q_out, None)
    T, H, dk = ks
    rows = pages = None
    if not (k.is_contiguous() and v.is_contiguous()):
        if k.numel() and (k.stride(2) != 1 or v.stride(2) != 1):
            raise ValueError("rows of k and v must be contiguous")
        rows = _strides(k, v)
    if not (k_cache.is_contiguous() and v_cache.is_contiguous()):
        if k_cache.numel() and (k_cache.stride(3) != 1 or v_cache.stride(3) != 1):
            raise ValueError("rows of a cache must be contiguous")
        pages = _strides(k_cache, v_cache)
    if plan is None:
        rc = L.gdn_paged_write(k.data_ptr(), v.data_ptr(), rows, k_cache.data_ptr(), v_cache.data_ptr(), pages,
                               slots.data_ptr(), T, H, dk, vs[2], cs[0], cs[2], dt, torch._C._cuda_getCurrentRawStream(dev))
        if rc != OK:
            raise GdnError(rc, "gdn_paged_write")
        return None
    qs, axes, ps = q.shape, plan.n_axes, positions.shape
    if not (len(qs) == 3 and qs[0] == T and qs[2] == dk and q.dtype is dtype and q.get_device() == dev and plan._dev == dev
            and positions.dtype is i32 and positions.get_device() == dev and positions.is_contiguous()
            and (ps == (axes, T) or (axes == 1 and ps == (T,)))
            and (q_out is None or (q_out.shape == qs and q_out.dtype is dtype and q_out.get_device() == dev))):
        _refuse((("q", q, (T, None, dk), dtype, dev), ("plan", plan.data, (plan.rot_dim // 2, 2), torch.int64, dev),
                 ("positions", positions, (T,) if len(ps) == 1 and axes == 1 else (axes, T), i32, dev),
                 ("q_out", q_out, tuple(qs), dtype, dev)))
    dense = q.is_contiguous()
    if q_out is None:
        q_out = torch.empty_like(q) if dense else torch.empty(qs, dtype=dtype, device=q.device)
    elif not q_out.is_contiguous():
        dense = False
    turned = None
    if not dense:
        if q.numel() and (q.stride(2) != 1 or q_out.stride(2) != 1):
            raise ValueError("rows of q and q_out must be contiguous")
        turned = _strides(q, q_out)
    rc = L.gdn_rotary_write(
        q.data_ptr(), q_out.data_ptr(), k.data_ptr(), v.data_ptr(), turned, rows, k_cache.data_ptr(), v_cache.data_ptr(),
        pages, positions.data_ptr(), plan._ptr, slots.data_ptr(), T, qs[1], H, dk, vs[2], plan.rot_dim, axes, cs[0], cs[2],
        plan._flags, dt, torch._C._cuda_getCurrentRawStream(dev))
    if rc != OK:
        raise GdnError(rc, "gdn_rotary_write")
    return q_out


def flash_attn_paged_supports(n_q: int, head_dim_k: int, head_dim_v: int) -> bool:
    """Whether ``flash_attn_paged`` serves this shape (fewer than 20 queries; widths each 64, 128 or 256)."""
    return bool(lib().gdn_flash_attn_paged_supports(int(n_q), int(head_dim_k), int(head_dim_v)))


def flash_attn_paged_workspace_bytes(n_seqs, n_heads, n_heads_kv, n_q, head_dim_k, head_dim_v, page_size, max_pages,
                                     dtype=None) -> int:
    """Bytes that ``flash_attn_paged`` needs as its ``workspace`` (0: none) for rows of ``dtype`` (default bf16)."""
    torch = _kv4_torch()
    return int(lib().gdn_flash_attn_paged_workspace_bytes(
        n_seqs, n_heads, n_heads_kv, n_q, head_dim_k, head_dim_v, page_size, max_pages,
        _kv4_dtype(torch.bfloat16 if dtype is None else dtype, "dtype")))


def flash_attn_paged(q, k_cache, v_cache, page_table, seq_lens, mask=None, scale=None, *, causal: bool = False,
                     out=None, out_dtype=None, workspace=None, stream=None):
    """Decode attention over a paged cache: out[b, i, h] = softmax_j(scale q[b,h,i] . k[b,hk,j] + mask[b,0,i,j])
    v[b,hk,j] over the seq_lens[b] tokens of each sequence (with ``causal``, j <= seq_lens[b] - n_q + i), hk = h //
    (n_heads / n_heads_kv).

    q: (n_seqs, n_heads, n_q, dk), any strides with contiguous, 16-byte aligned rows; k_cache, v_cache: (n_pages,
    n_heads_kv, page_size, dk / dv) of q's dtype (fp32, bf16 or fp16); page_table (n_seqs, max_pages) and seq_lens
    (n_seqs) int32; mask: (n_seqs, 1, n_q, max_pages * page_size) of q's dtype, additive, or None; scale defaults
    to 1/sqrt(dk).  Returns out (n_seqs, n_q, n_heads, dv) of ``out_dtype`` (fp32 by default, or a given out's
    dtype).  Rows that see no token are zeros; tokens that a row does not see have no effect on it.
    ``workspace``: an optional uint8 CUDA tensor of flash_attn_paged_workspace_bytes(...) bytes for one call at a
    time; without it the library allocates in stream order."""
    L, torch = _lib or lib(), _torch or _kv4_torch()
    dtype, dev, qs, cs, vs, ts, i32 = (q.dtype, q.get_device(), q.shape, k_cache.shape, v_cache.shape, page_table.shape,
                                       torch.int32)
    dt = _KV4_DTYPES.get(dtype)
    if dt is None:
        _kv4_dtype(dtype, "q")
    if not (dev >= 0 and len(qs) == 4 and len(cs) == 4 and len(vs) == 4 and len(ts) == 2
            and cs[0] == vs[0] and cs[1] == vs[1] and cs[2] == vs[2] and qs[3] == cs[3] and ts[0] == qs[0]
            and k_cache.dtype is dtype and v_cache.dtype is dtype
            and k_cache.get_device() == dev and v_cache.get_device() == dev
            and page_table.dtype is i32 and page_table.get_device() == dev and page_table.is_contiguous()
            and seq_lens.shape == (qs[0],) and seq_lens.dtype is i32 and seq_lens.get_device() == dev
            and seq_lens.is_contiguous()):
        _refuse((("q", q, (None, None, None, cs[-1]), dtype, dev), ("k_cache", k_cache, (None,) * 4, dtype, dev),
                 ("v_cache", v_cache, tuple(cs[:3]) + (None,), dtype, dev),
                 ("page_table", page_table, (qs[0], None), i32, dev), ("seq_lens", seq_lens, (qs[0],), i32, dev)))
    if stream is not None or torch._C._cuda_getDevice() != dev:
        return _there(dev, stream, flash_attn_paged, q, k_cache, v_cache, page_table, seq_lens, mask, scale, causal=causal,
                      out=out, out_dtype=out_dtype, workspace=workspace)
    B, H, n_q, dk = qs
    n_pages, Hkv, page, dv = vs
    rows = pages = None
    if not q.is_contiguous():
        if q.numel() and q.stride(3) != 1:
            raise ValueError("rows of q must be contiguous")
        rows = _strides(q)
    if not (k_cache.is_contiguous() and v_cache.is_contiguous()):
        if k_cache.numel() and (k_cache.stride(3) != 1 or v_cache.stride(3) != 1):
            raise ValueError("rows of a cache must be contiguous")
        pages = _strides(k_cache, v_cache)
    mask_at = ws_at = None
    ws_bytes = 0
    if mask is not None:
        if mask.shape != (B, 1, n_q, ts[1] * page) or mask.dtype is not dtype or mask.get_device() != dev \
                or not mask.is_contiguous():
            raise ValueError(f"mask: expected contiguous {(B, 1, n_q, ts[1] * page)} {dtype} on the tensors' device, got "
                             f"{tuple(mask.shape)} {mask.dtype}")
        mask_at = mask.data_ptr()
    if workspace is not None:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous and on the tensors' device")
        ws_at, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    if out is None:
        if out_dtype is None:
            out_dtype = torch.float32
        out = torch.empty((B, n_q, H, dv), dtype=out_dtype, device=q.device)
    elif out.shape != (B, n_q, H, dv) or (out_dtype is not None and out.dtype != out_dtype) or not out.is_contiguous() \
            or out.get_device() != dev:
        raise ValueError(f"out must be contiguous {(B, n_q, H, dv)} {out_dtype or ''} on the tensors' device")
    odt = _KV4_DTYPES.get(out.dtype)
    if odt is None:
        _kv4_dtype(out.dtype, "out_dtype")
    rc = L.gdn_flash_attn_paged(
        q.data_ptr(), rows, k_cache.data_ptr(), v_cache.data_ptr(), pages, page_table.data_ptr(), seq_lens.data_ptr(),
        mask_at, out.data_ptr(), B, H, Hkv, n_q, dk, dv, n_pages, page, ts[1], dk ** -0.5 if scale is None else scale,
        1 if causal else 0, dt, odt, ws_at, ws_bytes, torch._C._cuda_getCurrentRawStream(dev))
    if rc != OK:
        raise GdnError(rc, "gdn_flash_attn_paged")
    return out
