"""ctypes binding of ``libmla_b200.so`` (declared in ``include/mla.h``).

The prompt calls, whose small sizes take less time than ten tensors' checks in Python, go
through the same checks in C++ (``csrc/marshal.cpp``) first; those decline what is not
exactly right, and the checks here then say what is wrong.  Without that module, or with one
that was built for another torch, the checks here are the only ones.

Argument marshalling only: every function here forwards torch tensors' device
pointers and sizes to the C ABI call of the same name and raises ``MlaError``
on a non-OK status.  There is no fallback: if the library is missing the
import fails.
"""

from __future__ import annotations

import ctypes
import dataclasses
import os
import warnings
from typing import Optional

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmla_b200.so")

MLA_BF16, MLA_FP32 = 0, 1
MLA_ROPE_INTERLEAVED, MLA_ROPE_HALF = 0, 1
MLA_CACHE_NATIVE, MLA_CACHE_INT8 = 0, 1
MLA_INT8_ROW_BYTES = 656

STATUS = {0: "MLA_OK", 1: "MLA_ERR_INVALID_ARG", 2: "MLA_ERR_UNSUPPORTED",
          3: "MLA_ERR_ALIGNMENT", 4: "MLA_ERR_WORKSPACE", 5: "MLA_ERR_CUDA",
          6: "MLA_ERR_DEVICE_RANGE", 7: "MLA_ERR_TIMEOUT"}

EXPORTS = ("mla_workspace_size", "mla_workspace_init", "mla_cache_append", "mla_absorb_q",
           "mla_decode_attn", "mla_decode_attn_partial", "mla_merge_partials",
           "mla_decode_attn_noalloc", "mla_unabsorb_out", "mla_prompt_workspace_size",
           "mla_prompt_append", "mla_cache_gather", "mla_prompt_attn",
           "mla_noalloc_get_device_error", "mla_get_device_error", "mla_debug_absorb_timeout",
           "mla_debug_prompt_timeout", "mla_status_string")


class MlaError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {STATUS.get(status, status)} ({status_string(status)})")


class _Dims(ctypes.Structure):
    _fields_ = [("n_heads", ctypes.c_int), ("d_c", ctypes.c_int), ("d_rope", ctypes.c_int),
                ("d_nope", ctypes.c_int), ("d_v", ctypes.c_int), ("page_size", ctypes.c_int),
                ("dtype", ctypes.c_int), ("rope_layout", ctypes.c_int),
                ("rope_base", ctypes.c_double), ("rms_eps", ctypes.c_double),
                ("softmax_scale", ctypes.c_double), ("cache_format", ctypes.c_int)]


class _Cache(ctypes.Structure):
    _fields_ = [("pool", ctypes.c_void_p), ("num_pages", ctypes.c_int),
                ("block_table", ctypes.c_void_p), ("max_pages_per_seq", ctypes.c_int),
                ("seq_lens", ctypes.c_void_p)]


class _Heads(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


@dataclasses.dataclass
class Dims:
    """Mirror of ``mla_dims``."""
    n_heads: int
    d_c: int
    d_rope: int
    d_nope: int
    d_v: int
    page_size: int
    dtype: int = MLA_BF16
    rope_layout: int = MLA_ROPE_INTERLEAVED
    rope_base: float = 10000.0
    rms_eps: float = 1e-6
    softmax_scale: float = 0.0
    cache_format: int = MLA_CACHE_NATIVE

    __slots__ = ("_kept", "__dict__", "__weakref__")     # (_kept is no field and not in __dict__)

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        if name != "_kept":
            object.__setattr__(self, "_kept", None)

    def c(self) -> _Dims:
        """A C struct of the fields."""
        return _Dims(self.n_heads, self.d_c, self.d_rope, self.d_nope, self.d_v, self.page_size,
                     self.dtype, self.rope_layout, self.rope_base, self.rms_eps,
                     self.softmax_scale, self.cache_format)

    def kept(self) -> _Dims:
        """The C struct for calls that only read it, made once; setting a field drops it."""
        k = self._kept
        if k is None:
            k = self.c()
            object.__setattr__(self, "_kept", k)
        return k

    @property
    def torch_dtype(self):
        return torch.bfloat16 if self.dtype == MLA_BF16 else torch.float32


@dataclasses.dataclass
class PagedCache:
    """Mirror of ``mla_paged_cache`` holding the torch tensors.

    pool ``[num_pages, page_size, d_c + d_rope]``, block_table
    ``[batch, max_pages_per_seq]`` int32, seq_lens ``[batch]`` int32 (None for
    the calls that do not read it).
    """
    pool: torch.Tensor
    block_table: torch.Tensor
    seq_lens: Optional[torch.Tensor]

    def c(self) -> _Cache:
        return _Cache(self.pool.data_ptr(), self.pool.shape[0], self.block_table.data_ptr(),
                      self.block_table.shape[1], _p(self.seq_lens))


_lib = None
_marshal = None


def lib() -> ctypes.CDLL:
    """Loads the library (raises if it has not been built)."""
    global _lib, _marshal
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: run `python -m mla_latent_kv_45_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        pd, pc = ctypes.POINTER(_Dims), ctypes.POINTER(_Cache)
        L.mla_workspace_size.argtypes = [pd, i, i, i, i]
        L.mla_workspace_size.restype = sz
        L.mla_workspace_init.argtypes = [vp, sz, vp]
        L.mla_cache_append.argtypes = [pd, pc, i, i, vp, vp, vp, vp, vp, vp, sz, vp]
        L.mla_absorb_q.argtypes = [pd, i, i, vp, vp, i, vp, vp, vp, vp, vp, vp, sz, vp]
        L.mla_decode_attn.argtypes = [pd, pc, i, vp, vp, vp, i, vp, sz, vp]
        L.mla_decode_attn_partial.argtypes = [pd, pc, i, vp, vp, vp, vp, i, vp, sz, vp]
        L.mla_merge_partials.argtypes = [pd, i, i, vp, vp, vp, vp, vp, vp]
        L.mla_decode_attn_noalloc.argtypes = [pd, pc, i, vp, vp, vp, i, vp]
        L.mla_unabsorb_out.argtypes = [pd, i, vp, vp, vp, i, vp, vp, sz, vp]
        i64, ph = ctypes.c_int64, ctypes.POINTER(_Heads)
        L.mla_prompt_workspace_size.argtypes = [pd, i, i]
        L.mla_prompt_workspace_size.restype = sz
        L.mla_prompt_append.argtypes = [pd, pc, i, i, vp, i, i64, vp, vp, vp, ph, ph, vp, sz, vp]
        L.mla_cache_gather.argtypes = [pd, pc, i, i, vp, vp, vp, vp, sz, vp]
        L.mla_prompt_attn.argtypes = [pd, i, i, i, i, ph, ph, ph, vp, i64, ph, vp, vp, vp, vp, vp,
                                      sz, vp]
        L.mla_get_device_error.argtypes = [vp, vp]
        L.mla_noalloc_get_device_error.argtypes = [vp]
        L.mla_debug_absorb_timeout.argtypes = [i, ctypes.c_uint]
        L.mla_debug_prompt_timeout.argtypes = [i, ctypes.c_uint]
        L.mla_status_string.argtypes = [i]
        L.mla_status_string.restype = ctypes.c_char_p
        for name in EXPORTS:
            if name not in ("mla_workspace_size", "mla_prompt_workspace_size",
                            "mla_status_string"):
                getattr(L, name).restype = i
        _marshal = _load_marshal(L)
        _lib = L
    return _lib


def torch_build() -> str:
    """The torch in use, as far as the binary interface of an extension goes."""
    return (f"{torch.__version__} {torch.version.git_version} "
            f"abi{int(torch._C._GLIBCXX_USE_CXX11_ABI)}")


def _load_marshal(L: ctypes.CDLL):
    """The prompt calls' checks in C++, or None."""
    try:
        from . import _marshal as m
        if m.BUILT_FOR != torch_build():
            raise ImportError(f"it was built for torch {m.BUILT_FOR}, this is {torch_build()}")
    except (ImportError, AttributeError) as e:
        warnings.warn("the prompt calls go through their checks in Python, which take the host "
                      f"some 10 us a call: no extension module _marshal ({e}); "
                      "`python -m mla_latent_kv_45_b200.build` builds it")
        return None
    m.bind(*(ctypes.cast(getattr(L, f), ctypes.c_void_p).value
             for f in ("mla_prompt_append", "mla_cache_gather", "mla_prompt_attn")))
    return m


def status_string(status: int) -> str:
    return lib().mla_status_string(status).decode()


def _p(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _ok(fn: str, st: int):
    if st != 0:
        raise MlaError(fn, st)


def mla_workspace_size(dims: Dims, batch: int, d_model: int, d_q: int, num_splits: int = 0) -> int:
    d = dims.c()
    return int(lib().mla_workspace_size(ctypes.byref(d), batch, d_model, d_q, num_splits))


def mla_workspace_init(ws: torch.Tensor, stream=None):
    _ok("mla_workspace_init", lib().mla_workspace_init(_p(ws), ws.numel() * ws.element_size(),
                                                       _stream(stream)))


def mla_cache_append(dims: Dims, cache: PagedCache, h, W_DKV, W_KR, gamma, positions,
                     ws: torch.Tensor, stream=None):
    d, c = dims.c(), cache.c()
    _ok("mla_cache_append", lib().mla_cache_append(
        ctypes.byref(d), ctypes.byref(c), h.shape[0], h.shape[1], _p(h), _p(W_DKV), _p(W_KR),
        _p(gamma), _p(positions), _p(ws), ws.numel() * ws.element_size(), _stream(stream)))


def mla_absorb_q(dims: Dims, x, W_DQ, W_UQ, W_QR, W_UK, positions, q_lat, ws: torch.Tensor,
                 stream=None):
    d = dims.c()
    d_q = W_DQ.shape[0] if W_DQ is not None else x.shape[1]
    _ok("mla_absorb_q", lib().mla_absorb_q(
        ctypes.byref(d), x.shape[0], x.shape[1], _p(x), _p(W_DQ), d_q, _p(W_UQ), _p(W_QR),
        _p(W_UK), _p(positions), _p(q_lat), _p(ws), ws.numel() * ws.element_size(),
        _stream(stream)))


def mla_decode_attn(dims: Dims, cache: PagedCache, q_lat, z, lse=None, num_splits: int = 0,
                    ws: torch.Tensor = None, stream=None):
    d, c = dims.c(), cache.c()
    _ok("mla_decode_attn", lib().mla_decode_attn(
        ctypes.byref(d), ctypes.byref(c), q_lat.shape[0], _p(q_lat), _p(z), _p(lse), num_splits,
        _p(ws), ws.numel() * ws.element_size(), _stream(stream)))


def mla_decode_attn_partial(dims: Dims, cache: PagedCache, q_lat, O, m, l, num_splits: int = 0,
                            ws: torch.Tensor = None, stream=None):
    """Unnormalised partial softmax (O, m, l) over the rows this cache holds."""
    d, c = dims.c(), cache.c()
    _ok("mla_decode_attn_partial", lib().mla_decode_attn_partial(
        ctypes.byref(d), ctypes.byref(c), q_lat.shape[0], _p(q_lat), _p(O), _p(m), _p(l),
        num_splits, _p(ws), ws.numel() * ws.element_size(), _stream(stream)))


def mla_merge_partials(dims: Dims, O, m, l, z, lse=None, stream=None):
    """z (and lse) from partials stacked as O [n, B, H, d_c], m and l [n, B, H]."""
    d = dims.c()
    _ok("mla_merge_partials", lib().mla_merge_partials(
        ctypes.byref(d), O.shape[1], O.shape[0], _p(O), _p(m), _p(l), _p(z), _p(lse),
        _stream(stream)))


def mla_decode_attn_noalloc(dims: Dims, cache: PagedCache, q_lat, z, lse=None,
                            num_splits: int = 0, stream=None):
    """Decode attention with the library's fixed internal scratch (no workspace)."""
    d, c = dims.c(), cache.c()
    _ok("mla_decode_attn_noalloc", lib().mla_decode_attn_noalloc(
        ctypes.byref(d), ctypes.byref(c), q_lat.shape[0], _p(q_lat), _p(z), _p(lse), num_splits,
        _stream(stream)))


def mla_unabsorb_out(dims: Dims, z, W_UV, W_O, out, ws: torch.Tensor, stream=None):
    d = dims.c()
    d_model = W_O.shape[0] if W_O is not None else 0
    _ok("mla_unabsorb_out", lib().mla_unabsorb_out(
        ctypes.byref(d), z.shape[0], _p(z), _p(W_UV), _p(W_O), d_model, _p(out), _p(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


# The checks below stand between a small call and its launch, so each looks at a
# tensor's attributes once.

def _bad(fn: str, name: str, t: torch.Tensor, want) -> ValueError:
    return ValueError(f"{fn}: {name} is {t.dtype} {tuple(t.shape)} with strides {t.stride()} on "
                      f"{t.device}; wanted {want}")


def _heads(fn: str, dtype, dev: int, t: torch.Tensor, name: str, tokens: int, heads: int,
           width: int) -> _Heads:
    """The view of a [tokens, heads, width] tensor (any token and head strides)."""
    st = t.stride()
    if (t.dtype is not dtype or t.shape != (tokens, heads, width) or st[2] != 1 and width > 1
            or t.get_device() != dev):
        raise _bad(fn, name, t, f"{dtype} [{tokens}, {heads}, {width}] on cuda:{dev}, last axis "
                                "contiguous")
    return _Heads(t.data_ptr(), st[0], st[1])


def _rows(fn: str, dtype, dev: int, t: torch.Tensor, name: str, rows: int, width: int):
    """Address and row stride of a [rows, width] tensor (any row stride)."""
    st = t.stride()
    if (t.dtype is not dtype or t.shape != (rows, width) or st[1] != 1 and width > 1
            or t.get_device() != dev):
        raise _bad(fn, name, t, f"{dtype} [{rows}, {width}] on cuda:{dev}, last axis contiguous")
    return t.data_ptr(), st[0]


def _dense(fn: str, dtype, dev: int, t: torch.Tensor, name: str, shape) -> int:
    """Address of a contiguous tensor of this type and shape."""
    if (t.dtype is not dtype or t.shape != shape or not t.is_contiguous()
            or t.get_device() != dev):
        raise _bad(fn, name, t, f"{dtype} {tuple(shape)} on cuda:{dev}, contiguous")
    return t.data_ptr()


def _device(fn: str, t: torch.Tensor) -> int:
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{fn}: tensors on {t.device}, not on a CUDA device")
    return dev


def _paged(fn: str, dims: Dims, dev: int, cache: PagedCache, batch: int) -> _Cache:
    if dims.cache_format == MLA_CACHE_INT8:
        width, dtype = MLA_INT8_ROW_BYTES, torch.uint8
    else:
        width, dtype = dims.d_c + dims.d_rope, dims.torch_dtype
    pages, table = cache.pool.shape[0], cache.block_table.shape[-1]
    return _Cache(_dense(fn, dtype, dev, cache.pool, "pool", (pages, dims.page_size, width)), pages,
                  _dense(fn, torch.int32, dev, cache.block_table, "block_table", (batch, table)),
                  table, None if cache.seq_lens is None else cache.seq_lens.data_ptr())


# The current stream's address without a Stream object around it, where torch has that.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _address(stream):
    """A given stream for the C++ checks: its address, of a stream that is on the current
    device (they take tensors of that device only); None stays None."""
    if stream is None:
        return None
    return stream.cuda_stream if stream.device_index == torch.cuda.current_device() else False


def _on(fn: str, dev: int, ws: torch.Tensor, stream) -> int:
    """The stream to launch on (default: the device's current one), after a look at ws."""
    if ws is None or ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError(f"{fn}: ws is not a contiguous tensor on cuda:{dev}")
    if stream is None:
        return _raw_stream(dev)
    if stream.device_index != dev:
        raise ValueError(f"{fn}: stream on {stream.device}, tensors on cuda:{dev}")
    return stream.cuda_stream


def _call(fn: str, dev: int, call, *args):
    """Calls the library with the tensors' device current."""
    if torch.cuda.current_device() == dev:
        st = call(*args)
    else:
        with torch.cuda.device(dev):
            st = call(*args)
    if st != 0:
        raise MlaError(fn, st)


def mla_prompt_workspace_size(dims: Dims, batch: int, n_tokens: int) -> int:
    d = dims.c()
    return int(lib().mla_prompt_workspace_size(ctypes.byref(d), batch, n_tokens))


def mla_prompt_append(dims: Dims, cache: PagedCache, x, gamma, cu_tokens, ctx_lens=None,
                      q_rope=None, q_out=None, ws: torch.Tensor = None, stream=None):
    """Packed rows into the paged cache, normalised and rotated, and the queries rotated.

    x ``[tokens, d_c + d_rope]`` (any row stride; fp32 or the dims' type), cu_tokens ``[batch + 1]`` int32,
    ctx_lens ``[batch]`` int32 or None, q_rope and q_out ``[tokens, n_heads,
    d_rope]`` (any token and head strides; q_out may be q_rope) or None.
    """
    fn = "mla_prompt_append"
    lib()
    if _marshal is not None and (s := _address(stream)) is not False:
        st = _marshal.append(dims.kept(), cache.pool, cache.block_table, x, gamma, cu_tokens,
                             ctx_lens, q_rope, q_out, ws, s)
        if st is not None:
            return _ok(fn, st)
    dt, i32 = dims.torch_dtype, torch.int32
    dev, n, batch = _device(fn, x), x.shape[0], cu_tokens.numel() - 1
    xd = x.dtype if x.dtype is torch.float32 else dt
    xp, xs = _rows(fn, xd, dev, x, "x", n, dims.d_c + dims.d_rope)
    if (q_rope is None) != (q_out is None):
        raise ValueError(f"{fn}: q_rope and q_out go together")
    q = qo = None
    if q_rope is not None:
        q = ctypes.byref(_heads(fn, dt, dev, q_rope, "q_rope", n, dims.n_heads, dims.d_rope))
        qo = ctypes.byref(_heads(fn, dt, dev, q_out, "q_out", n, dims.n_heads, dims.d_rope))
    handle = _on(fn, dev, ws, stream)
    _call(fn, dev, lib().mla_prompt_append, ctypes.byref(dims.c()),
            ctypes.byref(_paged(fn, dims, dev, cache, batch)), batch, n, xp,
            MLA_FP32 if xd is torch.float32 else MLA_BF16, xs,
            _dense(fn, dt, dev, gamma, "gamma", (dims.d_c,)),
            _dense(fn, i32, dev, cu_tokens, "cu_tokens", (batch + 1,)),
            None if ctx_lens is None else _dense(fn, i32, dev, ctx_lens, "ctx_lens", (batch,)),
            q, qo, ws.data_ptr(), ws.nbytes, handle)


def mla_cache_gather(dims: Dims, cache: PagedCache, cu_rows, first_rows, rows,
                     ws: torch.Tensor = None, stream=None):
    """rows ``[n, d_c + d_rope]``: each sequence's cached rows from first_rows[b] (None: 0) on,
    packed at cu_rows ``[batch + 1]``; int8 rows come back as the values they hold."""
    fn = "mla_cache_gather"
    lib()
    if _marshal is not None and (s := _address(stream)) is not False:
        st = _marshal.gather(dims.kept(), cache.pool, cache.block_table, cu_rows, first_rows, rows,
                             ws, s)
        if st is not None:
            return _ok(fn, st)
    i32 = torch.int32
    dev, n, batch = _device(fn, rows), rows.shape[0], cu_rows.numel() - 1
    handle = _on(fn, dev, ws, stream)
    _call(fn, dev, lib().mla_cache_gather, ctypes.byref(dims.c()),
            ctypes.byref(_paged(fn, dims, dev, cache, batch)), batch, n,
            _dense(fn, i32, dev, cu_rows, "cu_rows", (batch + 1,)),
            None if first_rows is None else _dense(fn, i32, dev, first_rows, "first_rows", (batch,)),
            _dense(fn, dims.torch_dtype, dev, rows, "rows", (n, dims.d_c + dims.d_rope)),
            ws.data_ptr(), ws.nbytes, handle)


def mla_prompt_attn(dims: Dims, q_nope, q_rope, k_nope, k_rope, v, cu_q, cu_k, out, lse=None,
                    ws: torch.Tensor = None, stream=None):
    """Causal attention over packed sequences.

    q_nope ``[n_q, n_heads, d_nope]``, q_rope ``[n_q, n_heads, d_rope]``, k_nope
    ``[n_k, n_kv_heads, d_nope]``, v ``[n_k, n_kv_heads, d_v]`` (any token and
    head strides), k_rope ``[n_k, d_rope]`` (any row stride), cu_q and cu_k
    ``[batch + 1]`` int32, out ``[n_q, n_heads, d_v]``, lse ``[n_q, n_heads]``
    fp32 or None.
    """
    fn = "mla_prompt_attn"
    lib()
    if _marshal is not None and (s := _address(stream)) is not False:
        st = _marshal.attn(dims.kept(), q_nope, q_rope, k_nope, k_rope, v, cu_q, cu_k, out, lse,
                           ws, s)
        if st is not None:
            return _ok(fn, st)
    dt, i32, H = dims.torch_dtype, torch.int32, dims.n_heads
    dev, n_q, n_k, off = _device(fn, q_nope), q_nope.shape[0], k_nope.shape[0], cu_q.shape
    n_kv = k_nope.shape[1]
    krp, krs = _rows(fn, dt, dev, k_rope, "k_rope", n_k, dims.d_rope)
    handle = _on(fn, dev, ws, stream)
    _call(fn, dev, lib().mla_prompt_attn, ctypes.byref(dims.c()), off[0] - 1, n_q,
            n_k, n_kv, ctypes.byref(_heads(fn, dt, dev, q_nope, "q_nope", n_q, H, dims.d_nope)),
            ctypes.byref(_heads(fn, dt, dev, q_rope, "q_rope", n_q, H, dims.d_rope)),
            ctypes.byref(_heads(fn, dt, dev, k_nope, "k_nope", n_k, n_kv, dims.d_nope)), krp, krs,
            ctypes.byref(_heads(fn, dt, dev, v, "v", n_k, n_kv, dims.d_v)),
            _dense(fn, i32, dev, cu_q, "cu_q", (off[0],)),
            _dense(fn, i32, dev, cu_k, "cu_k", (off[0],)),
            _dense(fn, dt, dev, out, "out", (n_q, H, dims.d_v)),
            None if lse is None else _dense(fn, torch.float32, dev, lse, "lse", (n_q, H)),
            ws.data_ptr(), ws.nbytes, handle)


def mla_noalloc_get_device_error(stream=None) -> int:
    """Synchronises the stream; returns (and clears) the device status of the last
    allocation-free decode-attention call on the current device."""
    return int(lib().mla_noalloc_get_device_error(_stream(stream)))


def mla_debug_absorb_timeout(enable: bool, wait_limit_us: int = 0):
    """Test hook: make the absorption kernel's q_C hand-off wait run out (see mla.h)."""
    _ok("mla_debug_absorb_timeout", lib().mla_debug_absorb_timeout(int(enable), wait_limit_us))


def mla_debug_prompt_timeout(enable: bool, wait_limit_us: int = 0):
    """Test hook: limit the prompt attention kernel's waits (see mla.h)."""
    _ok("mla_debug_prompt_timeout", lib().mla_debug_prompt_timeout(int(enable), wait_limit_us))


def mla_get_device_error(ws: torch.Tensor, stream=None) -> int:
    """Synchronises the stream; returns the device status code (0 = OK) and clears it."""
    return int(lib().mla_get_device_error(_p(ws), _stream(stream)))
