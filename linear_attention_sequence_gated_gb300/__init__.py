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
           "gdn_kv4_read", "gdn_flash_attn_kv4", "gdn_flash_attn_kv4_workspace_bytes"]

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
