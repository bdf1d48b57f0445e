"""Python binding of libqmm, the gfx950 GGUF block-quantized matrix product.

Argument marshalling only: every function named ``qmm_*`` forwards to the C
function of the same name in ``libqmm.so`` (declared in ``include/qmm.h`` and
``include/qmm_probe.h`` and ``include/qmm_kv.h``).
Device buffers may be passed as torch tensors (their ``data_ptr()`` is used)
or as integer device addresses; ``stream`` defaults to torch's current
stream.  The ``qmm_*`` functions return the C status code.  The helpers
below them (``quantize_act``, ``dequantize``, ``mul_mat`` ...) allocate their
outputs with torch and raise :class:`QmmError` on a non-zero status.  The
key-value cache has three plain holders of tensors (:class:`KVCache`,
:class:`KVBatch`, :class:`Rope`) and the helpers :func:`kv_append` and
:func:`attn` on them.

There is no fallback: if ``libqmm.so`` is missing, loading fails loudly.
"""
from __future__ import annotations

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libqmm.so")

QMM_Q4_0, QMM_Q8_0, QMM_Q4_K, QMM_Q6_K, QMM_Q8_K, QMM_Q5_0 = 1, 2, 3, 4, 5, 6
QMM_OK, QMM_ERR_TYPE, QMM_ERR_SHAPE, QMM_ERR_NULL = 0, -1, -2, -3
QMM_ERR_ALIGN, QMM_ERR_UNSUPPORTED, QMM_ERR_HIP = -4, -5, -6

QMM_F32, QMM_F16, QMM_BF16 = 32, 33, 34
QMM_ROPE_PAIRS, QMM_ROPE_HALVES = 0, 1

TYPES = {"Q4_0": QMM_Q4_0, "Q8_0": QMM_Q8_0, "Q4_K": QMM_Q4_K, "Q6_K": QMM_Q6_K, "Q8_K": QMM_Q8_K,
         "Q5_0": QMM_Q5_0}

_lib = None


class qmm_kv_cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("type", ctypes.c_int32), ("n_kv", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32), ("n_pages", ctypes.c_int64)]


class qmm_kv_batch(ctypes.Structure):
    _fields_ = [("q_start", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("n_seqs", ctypes.c_int32), ("table_width", ctypes.c_int32), ("n_tokens", ctypes.c_int64),
                ("max_kv", ctypes.c_int64)]


class qmm_rope(ctypes.Structure):
    _fields_ = [("freqs", ctypes.c_void_p), ("pos", ctypes.c_void_p), ("n_rot", ctypes.c_int32),
                ("pairing", ctypes.c_int32), ("n_axes", ctypes.c_int32), ("sections", ctypes.c_int32 * 4)]


class qmm_attn_opts(ctypes.Structure):
    _fields_ = [("scale", ctypes.c_float), ("softcap", ctypes.c_float), ("window", ctypes.c_int32),
                ("algo", ctypes.c_int32), ("slopes", ctypes.c_void_p), ("prefix", ctypes.c_void_p)]


class QmmError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {qmm_strerror(code)} ({code})")
        self.code = code


def lib() -> ctypes.CDLL:
    """Load libqmm.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m block_quantized_amd.build` "
                               "(or __graft_entry__.build()); there is no fallback implementation")
        L = ctypes.CDLL(LIB_PATH)
        I, I64, P, SZ = ctypes.c_int, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
        sig = {
            "qmm_block_size": (I, [I]),
            "qmm_block_bytes": (SZ, [I]),
            "qmm_row_bytes": (SZ, [I, I64]),
            "qmm_vec_dot_type": (I, [I]),
            "qmm_quantize_act": (I, [I, P, P, I64, I64, P]),
            "qmm_quantize": (I, [I, P, P, I64, I64, P]),
            "qmm_dequantize": (I, [I, P, P, I64, I64, P]),
            "qmm_mul_mat": (I, [I, P, P, P, I64, I64, I64, P]),
            "qmm_mul_mat_algo": (I, [I, P, P, P, I64, I64, I64, I, P]),
            "qmm_mul_mat_multi": (I, [I, I, P, P, P, P, I, I64, I64, P]),
            "qmm_mul_mat_choice": (I, [I, I64, I64, I64]),
            "qmm_kv_bytes": (SZ, [I, I, I, I, I64]),
            "qmm_rope_freqs": (I, [P, I, ctypes.c_double, ctypes.c_double, P, P]),
            "qmm_kv_append": (I, [P, P, P, I, P, I64, P, I64, P, I64, I, P, P]),
            "qmm_attn": (I, [P, P, P, I, P, I64, I, P, P, SZ, P]),
            "qmm_attn_work": (SZ, [P, P, P, I, I]),
            "qmm_attn_choice": (I, [P, P, I, I]),
            "qmm_strerror": (ctypes.c_char_p, [I]),
            "qmm_probe_read": (I, [P, I64, P, I, P]),
            "qmm_probe_mfma": (I, [I, I64, P, P]),
            "qmm_probe_mfma_ops": (I64, [I, I64]),
            "qmm_probe_mfma16": (I, [I, I64, P, P]),
            "qmm_probe_mfma16_ops": (I64, [I, I64]),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _lib = L
    return _lib


EXPORTED = ("qmm_block_size", "qmm_block_bytes", "qmm_row_bytes", "qmm_vec_dot_type", "qmm_quantize_act",
            "qmm_quantize", "qmm_dequantize", "qmm_mul_mat", "qmm_mul_mat_algo", "qmm_mul_mat_multi",
            "qmm_mul_mat_choice", "qmm_kv_bytes", "qmm_rope_freqs", "qmm_kv_append", "qmm_attn", "qmm_attn_work",
            "qmm_attn_choice",
            "qmm_strerror", "qmm_probe_read", "qmm_probe_mfma", "qmm_probe_mfma_ops",
            "qmm_probe_mfma16", "qmm_probe_mfma16_ops")


def _ptr(a):
    if a is None:
        return None
    if isinstance(a, int):
        return a
    return a.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# ------------------------------------------------------------ C-ABI names

def qmm_block_size(t: int) -> int:
    return lib().qmm_block_size(t)


def qmm_block_bytes(t: int) -> int:
    return lib().qmm_block_bytes(t)


def qmm_row_bytes(t: int, K: int) -> int:
    return lib().qmm_row_bytes(t, K)


def qmm_vec_dot_type(wtype: int) -> int:
    return lib().qmm_vec_dot_type(wtype)


def qmm_quantize_act(dst, x, xq, N, K, stream=None) -> int:
    return lib().qmm_quantize_act(dst, _ptr(x), _ptr(xq), N, K, _stream(stream))


def qmm_quantize(dst, x, out, rows, K, stream=None) -> int:
    return lib().qmm_quantize(dst, _ptr(x), _ptr(out), rows, K, _stream(stream))


def qmm_dequantize(t, blocks, out, rows, K, stream=None) -> int:
    return lib().qmm_dequantize(t, _ptr(blocks), _ptr(out), rows, K, _stream(stream))


def qmm_mul_mat(wtype, W, xq, y, M, N, K, stream=None) -> int:
    return lib().qmm_mul_mat(wtype, _ptr(W), _ptr(xq), _ptr(y), M, N, K, _stream(stream))


def qmm_mul_mat_algo(wtype, W, xq, y, M, N, K, algo, stream=None) -> int:
    return lib().qmm_mul_mat_algo(wtype, _ptr(W), _ptr(xq), _ptr(y), M, N, K, algo, _stream(stream))


def qmm_mul_mat_choice(wtype, M, N, K) -> int:
    return lib().qmm_mul_mat_choice(wtype, M, N, K)


def qmm_mul_mat_multi(wtype, count, W, y, M, x, x_is_f32, N, K, stream=None) -> int:
    """W, y: sequences of `count` device buffers (tensors or addresses); M: row counts."""
    Wa = (ctypes.c_void_p * max(count, 1))(*[_ptr(w) for w in W[:count]]) if W is not None else None
    ya = (ctypes.c_void_p * max(count, 1))(*[_ptr(t) for t in y[:count]]) if y is not None else None
    Ma = (ctypes.c_int64 * max(count, 1))(*M[:count]) if M is not None else None
    return lib().qmm_mul_mat_multi(wtype, count, Wa, ya, Ma, _ptr(x), int(bool(x_is_f32)), N, K, _stream(stream))


def _ref(struct):
    return None if struct is None else ctypes.byref(struct)


def qmm_kv_bytes(t, n_kv, head_dim, page_size, n_pages) -> int:
    return lib().qmm_kv_bytes(t, n_kv, head_dim, page_size, n_pages)


def qmm_rope_freqs(freqs, n_rot, base, scale=1.0, factors=None, stream=None) -> int:
    return lib().qmm_rope_freqs(_ptr(freqs), n_rot, base, scale, _ptr(factors), _stream(stream))


def qmm_kv_append(cache, batch, rope, xtype, k, ldk, v, ldv, q, ldq, n_q, q_out, stream=None) -> int:
    """cache, batch, rope: the structures of the same C names (or None)."""
    return lib().qmm_kv_append(_ref(cache), _ref(batch), _ref(rope), xtype, _ptr(k), ldk, _ptr(v), ldv, _ptr(q), ldq,
                               n_q, _ptr(q_out), _stream(stream))


def qmm_attn(cache, batch, opts, xtype, q, ldq, n_q, out, work, work_bytes, stream=None) -> int:
    return lib().qmm_attn(_ref(cache), _ref(batch), _ref(opts), xtype, _ptr(q), ldq, n_q, _ptr(out), _ptr(work),
                          work_bytes, _stream(stream))


def qmm_attn_work(cache, batch, opts, xtype, n_q) -> int:
    return lib().qmm_attn_work(_ref(cache), _ref(batch), _ref(opts), xtype, n_q)


def qmm_attn_choice(cache, batch, xtype, n_q) -> int:
    return lib().qmm_attn_choice(_ref(cache), _ref(batch), xtype, n_q)


def qmm_probe_read(src, nbytes, sink, workgroups=0, stream=None) -> int:
    return lib().qmm_probe_read(_ptr(src), nbytes, _ptr(sink), workgroups, _stream(stream))


def qmm_probe_mfma(workgroups, iters, sink, stream=None) -> int:
    return lib().qmm_probe_mfma(workgroups, iters, _ptr(sink), _stream(stream))


def qmm_probe_mfma_ops(workgroups, iters) -> int:
    return lib().qmm_probe_mfma_ops(workgroups, iters)


def qmm_probe_mfma16(workgroups, iters, sink, stream=None) -> int:
    return lib().qmm_probe_mfma16(workgroups, iters, _ptr(sink), _stream(stream))


def qmm_probe_mfma16_ops(workgroups, iters) -> int:
    return lib().qmm_probe_mfma16_ops(workgroups, iters)


def qmm_strerror(code: int) -> str:
    return lib().qmm_strerror(code).decode()


# ------------------------------------------------------ allocating helpers

def _check(code: int, what: str):
    if code != QMM_OK:
        raise QmmError(code, what)


def quantize(dst: int, x, stream=None):
    """fp32 (rows, K) CUDA tensor -> (rows, row_bytes) uint8 tensor of dst blocks."""
    import torch
    rows, K = x.shape
    out = torch.empty((rows, qmm_row_bytes(dst, K)), dtype=torch.uint8, device=x.device)
    _check(qmm_quantize(dst, x, out, rows, K, stream), "qmm_quantize")
    return out


def quantize_act(dst: int, x, stream=None):
    import torch
    rows, K = x.shape
    out = torch.empty((rows, qmm_row_bytes(dst, K)), dtype=torch.uint8, device=x.device)
    _check(qmm_quantize_act(dst, x, out, rows, K, stream), "qmm_quantize_act")
    return out


def dequantize(t: int, blocks, rows: int, K: int, stream=None):
    import torch
    out = torch.empty((rows, K), dtype=torch.float32, device=blocks.device)
    _check(qmm_dequantize(t, blocks, out, rows, K, stream), "qmm_dequantize")
    return out


def mul_mat_multi(wtype: int, Ws, Ms, x, N: int, K: int, x_is_f32: bool = False, stream=None):
    """Several matrices sharing x in one launch -> list of (N, M_i) outputs."""
    import torch
    ys = [torch.empty((N, M), dtype=torch.float32, device=x.device) for M in Ms]
    _check(qmm_mul_mat_multi(wtype, len(Ws), Ws, ys, list(Ms), x, x_is_f32, N, K, stream), "qmm_mul_mat_multi")
    return ys


def mul_mat(wtype: int, W, xq, M: int, N: int, K: int, algo: int = 0, stream=None):
    import torch
    y = torch.empty((N, M), dtype=torch.float32, device=W.device)
    _check(qmm_mul_mat_algo(wtype, W, xq, y, M, N, K, algo, stream), "qmm_mul_mat")
    return y


# ---------------------------------------------------- the key-value cache
#
# A step of a small model is launches of a few microseconds, so these helpers
# look at each tensor once and as cheaply as torch allows.

_torch = None  # torch, once a helper below has needed it
_raw_stream = None  # device index -> handle of its current stream


def _need_torch():
    global _torch, _raw_stream
    if _torch is None:
        import torch
        # a tenth of a microsecond instead of the two that a Stream object takes
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda dev: torch.cuda.current_stream(dev).cuda_stream)
        _torch = torch
    return _torch


def _refuse(code: int, what: str):
    raise QmmError(code, what)


def _device_of(what: str, *tensors) -> int:
    """The index of the one GPU that all the tensors (None left out) lie on."""
    devs = {t.get_device() for t in tensors if t is not None}
    if len(devs) != 1 or min(devs) < 0:
        _refuse(QMM_ERR_UNSUPPORTED, f"{what}: tensors have to lie on one GPU")
    return devs.pop()


def _elsewhere(dev: int, stream):
    """(stream handle, context) for a stream given by the caller, or another
    device than the current one: allocations and launches within the context
    belong to that stream of that device."""
    torch = _need_torch()
    if stream is None:
        return torch.cuda.current_stream(dev).cuda_stream, torch.cuda.device(dev)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=dev) if stream else torch.cuda.default_stream(dev)
    if stream.device.index != dev:
        _refuse(QMM_ERR_UNSUPPORTED, "the stream belongs to another device than the tensors")
    return stream.cuda_stream, torch.cuda.stream(stream)


def _int32(what: str, t, *shape):
    if t.dtype != _need_torch().int32 or not t.is_contiguous() or tuple(t.shape) != shape:
        _refuse(QMM_ERR_SHAPE, f"{what}: a contiguous int32 tensor of shape {shape} is wanted")


class KVCache:
    """The paged cache of one layer: tensors k and v of n_pages x n_kv x
    page_size rows (Q8_0 blocks as uint8, float16 or bfloat16, or the bytes of
    these as uint8; see qmm_kv.h)."""

    def __init__(self, k, v, type: int, n_kv: int, head_dim: int, page_size: int):
        page = qmm_kv_bytes(type, n_kv, head_dim, page_size, 1)
        if not page or max(type, n_kv, head_dim, page_size) >= 1 << 31:  # (ctypes took their low 32 bits)
            _refuse(QMM_ERR_UNSUPPORTED, "KVCache: type, heads, head_dim or page_size")
        size = k.numel() * k.element_size()
        if size != v.numel() * v.element_size() or not size or size % page:
            _refuse(QMM_ERR_SHAPE, f"KVCache: k and v have to be whole pages of {page} bytes, as many of each")
        if not k.is_contiguous() or not v.is_contiguous():
            _refuse(QMM_ERR_UNSUPPORTED, "KVCache: k and v have to be contiguous")
        torch = _need_torch()
        own = {QMM_F16: torch.float16, QMM_BF16: torch.bfloat16}.get(type, torch.uint8)
        if k.dtype not in (own, torch.uint8) or v.dtype not in (own, torch.uint8):
            _refuse(QMM_ERR_UNSUPPORTED, f"KVCache: k and v have to hold {own} values, or bytes (uint8)")
        self.dev = _device_of("KVCache", k, v)
        self.k, self.v, self.type = k, v, type
        self.n_kv, self.head_dim, self.page_size, self.n_pages = n_kv, head_dim, page_size, size // page
        self.c = qmm_kv_cache(k.data_ptr(), v.data_ptr(), type, n_kv, head_dim, page_size, self.n_pages)
        self.ref = ctypes.byref(self.c)

    @classmethod
    def allocate(cls, type: int, n_kv: int, head_dim: int, page_size: int, n_pages: int, device="cuda"):
        """A cache of n_pages pages, contents undefined."""
        torch = _need_torch()
        if not qmm_kv_bytes(type, n_kv, head_dim, page_size, n_pages):
            _refuse(QMM_ERR_UNSUPPORTED, "KVCache.allocate: type, heads, head_dim, page_size or n_pages")
        dtype = {QMM_Q8_0: torch.uint8, QMM_F16: torch.float16, QMM_BF16: torch.bfloat16}[type]
        row = qmm_row_bytes(QMM_Q8_0, head_dim) if type == QMM_Q8_0 else head_dim
        k, v = (torch.empty((n_pages, n_kv, page_size, row), dtype=dtype, device=device) for _ in range(2))
        return cls(k, v, type, n_kv, head_dim, page_size)


class KVBatch:
    """The new tokens of a batch: q_start (n_seqs + 1), kv_len (n_seqs), table
    (n_seqs x width), int32 on the GPU, and the rows of q, k and v."""

    def __init__(self, q_start, kv_len, table, n_tokens: int, max_kv: int = 0):
        n = kv_len.numel()
        if not 0 < n_tokens < 1 << 23 or max_kv < 0:
            _refuse(QMM_ERR_SHAPE, "KVBatch: n_tokens has to be 1 to 2^23 - 1, max_kv 0 or more")
        max_kv = min(max_kv, 1 << 30)
        _int32("KVBatch: kv_len", kv_len, n)
        _int32("KVBatch: q_start", q_start, n + 1)
        if table.dim() != 2:
            _refuse(QMM_ERR_SHAPE, "KVBatch: table has to be n_seqs x width")
        _int32("KVBatch: table", table, n, table.shape[1])
        self.dev = _device_of("KVBatch", q_start, kv_len, table)
        self.q_start, self.kv_len, self.table, self.n_tokens, self.n_seqs = q_start, kv_len, table, n_tokens, n
        self.c = qmm_kv_batch(q_start.data_ptr(), kv_len.data_ptr(), table.data_ptr(), n, table.shape[1], n_tokens,
                              max_kv)
        self.ref = ctypes.byref(self.c)


class Rope:
    """The rotation of positions: freqs (float64, n_rot / 2, from
    :func:`rope_freqs`), the pairing, and pos (int32, axes x tokens, or None
    for the index in the sequence) with the pairs of each axis."""

    def __init__(self, freqs, pairing: int, pos=None, sections=None):
        if freqs.dtype != _need_torch().float64 or not freqs.is_contiguous() or freqs.dim() != 1:
            _refuse(QMM_ERR_SHAPE, "Rope: freqs has to be a contiguous float64 vector")
        if pairing not in (QMM_ROPE_PAIRS, QMM_ROPE_HALVES):
            _refuse(QMM_ERR_UNSUPPORTED, "Rope: pairing has to be QMM_ROPE_PAIRS or QMM_ROPE_HALVES")
        axes = len(sections) if sections is not None else 1
        if not 1 <= axes <= 4:
            _refuse(QMM_ERR_SHAPE, "Rope: 1 to 4 axes")
        if sections is not None and not all(0 <= n <= freqs.numel() for n in sections):  # ctypes would cut them
            _refuse(QMM_ERR_SHAPE, "Rope: the pairs of the axes have to be those of freqs")
        if pos is not None:
            if pos.dim() == 1:
                pos = pos[None]
            if pos.dim() != 2:
                _refuse(QMM_ERR_SHAPE, "Rope: pos has to be axes x tokens")
            _int32("Rope: pos", pos, axes, pos.shape[1])
        self.dev = _device_of("Rope", freqs, pos)
        self.freqs, self.pos = freqs, pos
        self.tokens = None if pos is None else pos.shape[1]
        parts = list(sections if sections is not None else []) + [0] * 4
        self.c = qmm_rope(freqs.data_ptr(), _ptr(pos), 2 * freqs.numel(), pairing, axes,
                          (ctypes.c_int32 * 4)(*parts[:4]))
        self.ref = ctypes.byref(self.c)


def rope_freqs(n_rot: int, base: float, scale: float = 1.0, factors=None, device="cuda", stream=None):
    """The angles per position of n_rot / 2 pairs, float64."""
    torch = _need_torch()
    dev = torch.device(device) if factors is None else factors.device
    if dev.type != "cuda":
        _refuse(QMM_ERR_UNSUPPORTED, "rope_freqs: a GPU is wanted")
    index = torch.cuda.current_device() if dev.index is None else dev.index
    if factors is not None and (factors.dtype != torch.float32 or factors.numel() != n_rot // 2
                                or not factors.is_contiguous()):
        _refuse(QMM_ERR_SHAPE, "rope_freqs: factors have to be n_rot / 2 contiguous float32 values")
    if not 0 < n_rot <= 65536:
        _refuse(QMM_ERR_SHAPE, "rope_freqs: n_rot has to be 2 to 65536")
    handle, where = _elsewhere(index, stream)
    with where:
        freqs = torch.empty(max(n_rot // 2, 1), dtype=torch.float64, device=torch.device("cuda", index))
        _check(qmm_rope_freqs(freqs, n_rot, base, scale, factors, handle), "qmm_rope_freqs")
    return freqs


def _token_rows(what: str, x, n_tokens: int, head_dim: int):
    """Checks a (tokens, heads, head_dim) activation, whose token rows may be
    apart, and gives (heads, that distance)."""
    shape = x.shape
    if len(shape) == 3 and shape[0] == n_tokens and shape[2] == head_dim and x.is_contiguous():
        return shape[1], shape[1] * head_dim
    if len(shape) != 3 or shape[0] != n_tokens or shape[2] != head_dim:
        _refuse(QMM_ERR_SHAPE, f"{what}: {n_tokens} x heads x {head_dim} is wanted")
    heads = shape[1]
    row, head, one = x.stride()
    if one != 1 or (head != head_dim and heads != 1):
        _refuse(QMM_ERR_UNSUPPORTED, f"{what}: the heads of a token have to lie one after another")
    return heads, row if n_tokens > 1 else heads * head_dim


def _xtype(what: str, dtype):
    if dtype == _torch.float32:
        return QMM_F32
    if dtype != _torch.bfloat16:
        _refuse(QMM_ERR_UNSUPPORTED, f"{what}: activations have to be float32 or bfloat16")
    return QMM_BF16


def _no_grad(what: str, *tensors):
    if _torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
        _refuse(QMM_ERR_UNSUPPORTED, f"{what}: no gradients are computed; detach the inputs or use torch.no_grad()")


def _new_out(x):
    return _torch.empty_like(x, memory_format=_torch.contiguous_format)


def kv_append(cache: KVCache, batch: KVBatch, k, v, q=None, rope=None, q_out=None, stream=None):
    """Stores k (rotated) and v (tokens, n_kv, head_dim) in the cache, and
    returns q (tokens, n_q, head_dim) rotated, in q_out if given.  No
    gradients: inputs that require them are refused where torch records them."""
    torch = _torch or _need_torch()
    dev, N, D, dtype = cache.dev, batch.n_tokens, cache.head_dim, k.dtype
    same = batch.dev == dev and k.get_device() == dev and v.get_device() == dev and v.dtype == dtype
    h, ldk = _token_rows("kv_append: k", k, N, D)
    h2, ldv = _token_rows("kv_append: v", v, N, D)
    if h != cache.n_kv or h2 != cache.n_kv:
        _refuse(QMM_ERR_SHAPE, f"kv_append: k and v have to have {cache.n_kv} heads")
    n_q = ldq = 0
    if q is not None:
        n_q, ldq = _token_rows("kv_append: q", q, N, D)
        same = same and q.get_device() == dev and q.dtype == dtype
    if q_out is not None:
        if q is None:
            _refuse(QMM_ERR_NULL, "kv_append: q_out without q")
        if q_out.shape != q.shape or not q_out.is_contiguous():
            _refuse(QMM_ERR_SHAPE, "kv_append: q_out has to be contiguous and of q's shape")
        same = same and q_out.get_device() == dev and q_out.dtype == dtype
    if rope is not None:
        same = same and rope.dev == dev
        if rope.tokens is not None and rope.tokens != N:
            _refuse(QMM_ERR_SHAPE, "kv_append: pos has to name a position for every token")
    if not same:
        _refuse(QMM_ERR_UNSUPPORTED, "kv_append: tensors have to lie on one GPU and be of one type")
    _no_grad("kv_append", k, v, q, q_out)
    xtype = _xtype("kv_append", dtype)
    if stream is not None or torch.cuda.current_device() != dev:
        handle, where = _elsewhere(dev, stream)
        with where:
            return _append(cache, batch, rope, xtype, k, ldk, v, ldv, q, ldq, n_q, q_out, handle)
    return _append(cache, batch, rope, xtype, k, ldk, v, ldv, q, ldq, n_q, q_out,
                   _raw_stream(dev))


def _append(cache, batch, rope, xtype, k, ldk, v, ldv, q, ldq, n_q, q_out, handle):
    if q is not None and q_out is None:
        q_out = _new_out(q)
    rc = lib().qmm_kv_append(cache.ref, batch.ref, None if rope is None else rope.ref, xtype, k.data_ptr(), ldk,
                             v.data_ptr(), ldv, _ptr(q), ldq, n_q, _ptr(q_out), handle)
    if rc != QMM_OK:
        raise QmmError(rc, "qmm_kv_append")
    return q_out


def attn(cache: KVCache, batch: KVBatch, q, scale=None, softcap: float = 0.0, window: int = 0, slopes=None,
         prefix=None, algo: int = 0, out=None, stream=None):
    """Attention of q (tokens, n_q, head_dim) over the cache -> (tokens, n_q,
    head_dim), in out if given.  scale defaults to head_dim ** -0.5.  Rows of
    no sequence are not written.  No gradients, as kv_append."""
    torch = _torch or _need_torch()
    dev, N, D, dtype = cache.dev, batch.n_tokens, cache.head_dim, q.dtype
    same = batch.dev == dev and q.get_device() == dev
    n_q, ldq = _token_rows("attn: q", q, N, D)
    if out is not None:
        if out.shape != q.shape or not out.is_contiguous():
            _refuse(QMM_ERR_SHAPE, "attn: out has to be contiguous and of q's shape")
        same = same and out.get_device() == dev and out.dtype == dtype
    if slopes is not None:
        if slopes.dtype != torch.float32 or slopes.numel() != n_q or not slopes.is_contiguous():
            _refuse(QMM_ERR_SHAPE, "attn: slopes have to be one contiguous float32 value a query head")
        same = same and slopes.get_device() == dev
    if prefix is not None:
        _int32("attn: prefix", prefix, batch.n_seqs)
        same = same and prefix.get_device() == dev
    if not same:
        _refuse(QMM_ERR_UNSUPPORTED, "attn: tensors have to lie on one GPU, and out be of q's type")
    if not 0 <= window < 1 << 31 or not 0 <= algo <= 2:  # ctypes would take their low 32 bits
        _refuse(QMM_ERR_UNSUPPORTED, "attn: window has to be 0 to 2^31 - 1, algo 0 to 2")
    _no_grad("attn", q, slopes, out)
    xtype = _xtype("attn", dtype)
    opts = ctypes.byref(qmm_attn_opts(D ** -0.5 if scale is None else scale, softcap, window, algo, _ptr(slopes),
                                      _ptr(prefix)))
    if stream is not None or torch.cuda.current_device() != dev:
        handle, where = _elsewhere(dev, stream)
        with where:
            return _attend(cache, batch, opts, xtype, q, ldq, n_q, out, handle)
    return _attend(cache, batch, opts, xtype, q, ldq, n_q, out, _raw_stream(dev))


def _attend(cache, batch, opts, xtype, q, ldq, n_q, out, handle):
    L = lib()
    need = L.qmm_attn_work(cache.ref, batch.ref, opts, xtype, n_q)
    if out is None:
        out = _new_out(q)
    work = _torch.empty(need, dtype=_torch.uint8, device=q.device) if need else None
    rc = L.qmm_attn(cache.ref, batch.ref, opts, xtype, q.data_ptr(), ldq, n_q, out.data_ptr(), _ptr(work), need,
                    handle)
    if rc != QMM_OK:
        raise QmmError(rc, "qmm_attn")
    return out
