"""bit_kv_cache_ott_gb300 -- Outlier Tokens Tracing (OTT) KV-cache quantization
on one GB300 GPU.

A thin ctypes binding over ``libott.so`` (C ABI in ``include/ott.h``): it only
marshals torch tensors into device pointers and streams. Every step of the
path (append, flush, prefill, decode attention) runs in the library's CUDA
kernels. There is no CPU fallback: if the library is missing or cannot load,
``load()`` raises.
"""
from __future__ import annotations

import array
import ctypes as C
import functools
import os

import torch

from . import synth  # noqa: F401  (seeded workloads)

__all__ = ["OTTCache", "ByteCache", "OTTError", "load", "status_str", "lib_path", "hbm_copy", "rope"]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "_build", "libott.so")
_lib = None

OTT_OK, OTT_ERR_INVALID, OTT_ERR_STATE, OTT_ERR_CAPACITY = 0, -1, -2, -3
OTT_ERR_OOM, OTT_ERR_CUDA, OTT_ERR_DEVICE = -4, -5, -6


class OTTError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {status_str(code)} ({code})")
        self.code = code


class StateExport(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in
                ("bidx", "kcode", "ks", "kz", "vcode", "vs", "vz", "tk", "tv", "pidx", "pnorm", "pk", "pv")]


class RopePlan(C.Structure):
    _fields_ = [("axes", C.c_int), ("sections", C.c_int * 4), ("base", C.c_double), ("interleaved", C.c_int),
                ("restart", C.c_int)]


SYMBOLS = ("ott_create", "ott_create_ragged", "ott_create_paged", "ott_release_seq", "ott_prefill_seq",
           "ott_free_blocks", "ott_create_cold", "ott_create_pct", "ott_export_cold", "ott_destroy", "ott_prefill", "ott_prefill_lens", "ott_append", "ott_step_host",
           "ott_decode_attn", "ott_decode_attn_static", "ott_decode_attn_topk",
           "ott_chunk_attn", "ott_append_chunk", "ott_decode_attn_window", "ott_rope", "ott_get_counts", "ott_get_seq_counts", "ott_block_count",
           "ott_export_state", "ott_check_device", "ott_device_bytes", "ott_status_str", "ott_hbm_copy", "ott_ex2_probe",
           "ott_byte_create", "ott_byte_destroy", "ott_byte_append", "ott_byte_append_seq", "ott_byte_read", "ott_byte_decode",
           "ott_byte_attn", "ott_byte_release", "ott_byte_reset", "ott_byte_counts", "ott_byte_free_blocks", "ott_byte_check",
           "ott_byte_bytes")


def lib_path() -> str:
    return _LIB_PATH


def load(build_if_missing: bool = False):
    """Load libott.so (raises if it is absent or broken)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        if not build_if_missing:
            raise RuntimeError(f"libott.so not built ({_LIB_PATH}); run __graft_entry__.build()")
        from .build import build
        build()
    L = C.CDLL(_LIB_PATH)
    P, i32, i64 = C.c_void_p, C.c_int, C.c_longlong
    L.ott_create.argtypes = [i32] * 8 + [C.POINTER(P)]
    L.ott_create_ragged.argtypes = [i32] * 8 + [C.POINTER(P)]
    L.ott_create_cold.argtypes = [i32] * 9 + [C.POINTER(P)]
    L.ott_create_pct.argtypes = [i32] * 10 + [C.POINTER(P)]
    L.ott_create_paged.argtypes = [i32] * 8 + [i64, C.POINTER(P)]
    L.ott_release_seq.argtypes = [P, i32, P]
    L.ott_prefill_seq.argtypes = [P, i32, P, P, i32, P]
    L.ott_free_blocks.argtypes = [P]
    L.ott_free_blocks.restype = i64
    L.ott_export_cold.argtypes = [P, i32, i32, P, P, P, P, P]
    L.ott_destroy.argtypes = [P]
    L.ott_prefill.argtypes = [P, P, P, i32, P]
    L.ott_prefill_lens.argtypes = [P, P, P, C.POINTER(i32), i32, P]
    L.ott_append.argtypes = [P, P, P, P]
    L.ott_step_host.argtypes = [P, P, P, P, P, i32, P]
    L.ott_decode_attn.argtypes = [P, P, P, P]
    L.ott_decode_attn_static.argtypes = [P, P, P, P]
    L.ott_decode_attn_topk.argtypes = [P, P, P, i32, P, P]
    L.ott_chunk_attn.argtypes = [P, P, P, P, P, i32, C.POINTER(i32), i32, i32, P]
    L.ott_append_chunk.argtypes = [P, P, P, i32, C.POINTER(i32), P]
    L.ott_decode_attn_window.argtypes = [P, P, P, i32, i32, P]
    L.ott_rope.argtypes = [P, P, i32, P, P, i32, P, i32, i32, i32, C.POINTER(RopePlan), P]
    L.ott_get_counts.argtypes = [P, C.POINTER(i64), C.POINTER(i32), C.POINTER(i32), C.POINTER(i32)]
    L.ott_get_seq_counts.argtypes = [P, i32, C.POINTER(i64), C.POINTER(i32), C.POINTER(i32), C.POINTER(i32)]
    L.ott_block_count.argtypes = [P, i32]
    L.ott_export_state.argtypes = [P, i32, i32, C.POINTER(StateExport)]
    L.ott_check_device.argtypes = [P]
    L.ott_device_bytes.argtypes = [P]
    L.ott_device_bytes.restype = i64
    L.ott_status_str.argtypes = [i32]
    L.ott_status_str.restype = C.c_char_p
    L.ott_hbm_copy.argtypes = [P, P, i64, P]
    L.ott_ex2_probe.argtypes = [P, P, i32, P]
    L.ott_byte_create.argtypes = [i32] * 7 + [i64, C.POINTER(P)]
    L.ott_byte_destroy.argtypes = [P]
    L.ott_byte_append.argtypes = [P, P, P, i32, P, P]
    L.ott_byte_append_seq.argtypes = [P, i32, P, P, i32, P]
    L.ott_byte_read.argtypes = [P, P, P, i32, i32, P]
    L.ott_byte_decode.argtypes = [P, P, P, i32, P, P]
    L.ott_byte_attn.argtypes = [P, P, P, P, P, i32, P, i32, P, P]
    L.ott_byte_release.argtypes = [P, i32, P]
    L.ott_byte_reset.argtypes = [P, P]
    L.ott_byte_counts.argtypes = [P, i32, C.POINTER(i64), C.POINTER(i32)]
    L.ott_byte_free_blocks.argtypes = [P]
    L.ott_byte_free_blocks.restype = i64
    L.ott_byte_check.argtypes = [P]
    L.ott_byte_bytes.argtypes = [P]
    L.ott_byte_bytes.restype = i64
    _lib = L
    return L


def status_str(code: int) -> str:
    return load().ott_status_str(code).decode()


def hbm_copy(dst: torch.Tensor, src: torch.Tensor, stream=None):
    """Copy src into dst (same byte size, CUDA tensors) with the library's
    streaming copy kernel: the bandwidth probe that times HBM in the same run
    as the decode."""
    if not (dst.is_cuda and src.is_cuda and dst.is_contiguous() and src.is_contiguous()):
        raise ValueError("hbm_copy: contiguous CUDA tensors")
    n = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() != n:
        raise ValueError("hbm_copy: sizes differ")
    _check(load().ott_hbm_copy(dst.data_ptr(), src.data_ptr(), n, _stream(stream)), "ott_hbm_copy")


def _check(rc: int, what: str):
    if rc != OTT_OK:
        raise OTTError(rc, what)


def _dev_ptr(t: torch.Tensor, shape, name) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.float16:
        raise TypeError(f"{name}: expected a CUDA float16 tensor")
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _stream(stream) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _new(make, stream, idx: int) -> torch.Tensor:
    """An output that a call makes itself, make(), for kernels on the given stream: made there if it is not the current
    one of device idx (whose freed memory may still be read, and whose fills may end late), and kept for the current
    one's reads."""
    if stream is None:
        return make()
    here = torch.cuda.current_stream(idx)
    if here.cuda_stream == stream.cuda_stream:
        return make()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device=idx)
    with torch.cuda.stream(stream):
        t = make()
    t.record_stream(here)
    return t


def rope(q: torch.Tensor | None, k: torch.Tensor | None, pos: torch.Tensor, sections, base: float = 10000.0,
         interleaved: bool = False, restart: bool = False, out_q: torch.Tensor | None = None,
         out_k: torch.Tensor | None = None, stream=None):
    """Rotary positions with len(sections) axes (ott_rope): q fp16 [B][Hq][n][d], k fp16 [B][Hkv][n][d] (either may be
    None), pos int32 [axes][B][n], all contiguous on one CUDA device. sections: the pairs of channels that turn with
    each axis; pair i is channels (i, half + i), half = sum(sections), or (2i, 2i + 1) if ``interleaved``; it turns by
    pos * base ** -e with e = i / half, or j / sections[a] for an axis's j-th pair if ``restart``. Outputs may be the
    inputs (in place). Returns (rotated q, rotated k), None for one that was not given."""
    x = k if q is None else q
    if x is None:
        raise ValueError("rope: q or k must be given")
    for t in (q, k):
        if t is not None and (not isinstance(t, torch.Tensor) or t.dim() != 4):
            raise ValueError("rope: expected [B][H][n][d] tensors")
    B, _, n, d = x.shape
    sections = tuple(map(int, sections))
    axes = len(sections)
    if not 1 <= axes <= 4:
        raise ValueError("rope: one to four axes")
    if not isinstance(pos, torch.Tensor) or not pos.is_cuda or pos.dtype != torch.int32:
        raise TypeError("pos: expected a CUDA int32 tensor")
    if pos.shape != (axes, B, n) or not pos.is_contiguous():
        raise ValueError(f"pos: expected contiguous shape {(axes, B, n)}, got {tuple(pos.shape)}")
    idx = x.get_device()
    qp, qo, out_q, Hq = _rope_operand(q, out_q, "q", B, n, d, stream)
    kp, ko, out_k, Hkv = _rope_operand(k, out_k, "k", B, n, d, stream)
    for t in (pos, q, k, out_q, out_k):
        if t is not None and t.get_device() != idx:
            raise ValueError(f"tensors on {t.device} and cuda:{idx}")
    if B and n and Hq + Hkv:
        plan = _rope_plan(sections, float(base), bool(interleaved), bool(restart))
        _on_device(idx, load().ott_rope, "ott_rope", qp, qo, Hq, kp, ko, Hkv, pos.data_ptr(), B, n, d, plan,
                   _stream_of(stream, idx))
    return out_q, out_k


def _rope_operand(x, out, name, B, n, d, stream):
    """(pointer, output's pointer, output, heads) of one of rope's tensors."""
    if x is None:
        if out is not None:
            raise ValueError(f"out_{name} without {name}")
        return None, None, None, 0
    H = x.shape[1]
    p = _dev_ptr(x, (B, H, n, d), name)
    if out is None:
        out = _new(lambda: torch.empty_like(x), stream, x.get_device())
        return p, out.data_ptr(), out, H
    return p, _dev_ptr(out, (B, H, n, d), f"out_{name}"), out, H


@functools.lru_cache(maxsize=64)
def _rope_plan(sections, base, interleaved, restart):
    sec = (C.c_int * 4)(*[_int32(x, "sections") for x in sections])
    return C.byref(RopePlan(len(sections), sec, base, int(interleaved), int(restart)))


def _int32(x, name: str) -> int:
    """x as the C ABI's int (ctypes would drop the bits that do not fit)."""
    x = int(x)
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{name}: {x} does not fit 32 bits")
    return x


def _same_device(idx, *tensors):
    for t in tensors:
        if t.get_device() != idx:
            raise ValueError(f"tensors on {t.device} and cuda:{idx}")


def _stream_of(stream, idx: int) -> int:
    """The raw stream to queue on: the given one, else device idx's current one."""
    return (torch.cuda.current_stream(idx) if stream is None else stream).cuda_stream


# (torch.cuda.current_stream and current_device without their objects and checks)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda idx: torch.cuda.current_stream(idx).cuda_stream)
_raw_device = getattr(torch._C, "_cuda_getDevice", lambda: torch.cuda.current_device())


def _on_device(idx: int, fn, what: str, *args):
    """fn(*args) with device idx current (a context manager per call costs more than most of these kernels)."""
    prev = torch.cuda.current_device()
    if prev == idx:
        rc = fn(*args)
    else:
        torch.cuda.set_device(idx)
        try:
            rc = fn(*args)
        finally:
            torch.cuda.set_device(prev)
    _check(rc, what)


class OTTCache:
    """One OTT cache (one attention layer): ``create/prefill/append/decode_attn/destroy``.
    ``ragged=True`` creates it with ``ott_create_ragged`` so that ``prefill_lens``
    can give every sequence its own length. ``cold=C`` creates it with
    ``ott_create_cold``: displaced pool tokens go to a first-in-first-out
    fp16 cold pool of C slots instead of the new block. ``pct=(p, n_oc)``
    creates it with ``ott_create_pct``: the channel-conditioned outlier
    criterion, p in units of 1/10000 over n_oc outlier channels."""

    def __init__(self, B, Hq, Hkv, d, G=128, R=32, P=32, max_tokens=8192, ragged=False, cold=None,
                 pool_blocks=None, pct=None):
        L = load()
        self.B, self.Hq, self.Hkv, self.d, self.G, self.R, self.P = B, Hq, Hkv, d, G, R, P
        self.max_tokens = max_tokens
        self.ragged = ragged
        self.cold = cold
        h = C.c_void_p()
        if pool_blocks is not None:
            self.ragged = True
            _check(L.ott_create_paged(B, Hq, Hkv, d, G, R, P, max_tokens, int(pool_blocks), C.byref(h)),
                   "ott_create_paged")
        elif pct is not None:
            if ragged or cold is not None:
                raise ValueError("the channel criterion takes sequences of one length and writes tokens back")
            _check(L.ott_create_pct(B, Hq, Hkv, d, G, R, P, int(pct[0]), int(pct[1]), max_tokens, C.byref(h)),
                   "ott_create_pct")
        elif cold is not None:
            if ragged:
                raise ValueError("the cold-pool policy takes sequences of one length")
            _check(L.ott_create_cold(B, Hq, Hkv, d, G, R, P, int(cold), max_tokens, C.byref(h)), "ott_create_cold")
        else:
            create = L.ott_create_ragged if ragged else L.ott_create
            _check(create(B, Hq, Hkv, d, G, R, P, max_tokens, C.byref(h)),
                   "ott_create_ragged" if ragged else "ott_create")
        self._h = h
        self._dev = torch.cuda.current_device()

    def close(self):
        if getattr(self, "_h", None) and self._h.value:
            load().ott_destroy(self._h)
            self._h = C.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    @property
    def handle(self) -> int:
        return self._h.value

    def prefill(self, K: torch.Tensor, V: torch.Tensor, stream=None):
        Lq = K.shape[2] if K.dim() == 4 else -1
        shp = (self.B, self.Hkv, Lq, self.d)
        _check(load().ott_prefill(self._h, _dev_ptr(K, shp, "K"), _dev_ptr(V, shp, "V"), Lq,
                                  _stream(stream)), "ott_prefill")

    def prefill_lens(self, K: torch.Tensor, V: torch.Tensor, lens, stream=None):
        """Ragged prefill: K, V [B][Hkv][Lmax][d]; sequence b takes its first lens[b] tokens."""
        Lmax = K.shape[2] if K.dim() == 4 else -1
        shp = (self.B, self.Hkv, Lmax, self.d)
        ln = (C.c_int * self.B)(*[int(x) for x in lens])
        if len(lens) != self.B:
            raise ValueError("lens must hold one length per sequence")
        _check(load().ott_prefill_lens(self._h, _dev_ptr(K, shp, "K"), _dev_ptr(V, shp, "V"), ln, Lmax,
                                       _stream(stream)), "ott_prefill_lens")

    def append(self, k: torch.Tensor, v: torch.Tensor, stream=None):
        shp = (self.B, self.Hkv, self.d)
        _check(load().ott_append(self._h, _dev_ptr(k, shp, "k"), _dev_ptr(v, shp, "v"),
                                 _stream(stream)), "ott_append")

    def step_host(self, k: torch.Tensor, v: torch.Tensor, q: torch.Tensor, out: torch.Tensor, topk: int = 0,
                  stream=None):
        """One step from pinned host memory: append k, v (fp16 [B][Hkv][d]) and
        decode q (fp16 [B][Hq][d]) into out (fp16 [B][Hq][d]), all pinned CPU
        tensors; the kernels read and write them in place (ott_step_host).
        topk >= 1 decodes with Top-K sparse access over that many blocks.
        out is complete when the stream has passed the step."""
        for name, t, shp in (("k", k, (self.B, self.Hkv, self.d)), ("v", v, (self.B, self.Hkv, self.d)),
                             ("q", q, (self.B, self.Hq, self.d)), ("out", out, (self.B, self.Hq, self.d))):
            if not isinstance(t, torch.Tensor) or t.is_cuda or t.dtype != torch.float16 or not t.is_pinned():
                raise TypeError(f"{name}: expected a pinned CPU float16 tensor")
            if tuple(t.shape) != shp or not t.is_contiguous():
                raise ValueError(f"{name}: expected contiguous shape {shp}, got {tuple(t.shape)}")
        _check(load().ott_step_host(self._h, k.data_ptr(), v.data_ptr(), q.data_ptr(), out.data_ptr(), int(topk),
                                    _stream(stream)), "ott_step_host")

    def decode_attn(self, q: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        shp = (self.B, self.Hq, self.d)
        qp = _dev_ptr(q, shp, "q")
        if out is None:
            out = _new(lambda: torch.empty_like(q), stream, q.get_device())
        _check(load().ott_decode_attn(self._h, qp, _dev_ptr(out, shp, "out"), _stream(stream)), "ott_decode_attn")
        return out

    def decode_attn_topk(self, q: torch.Tensor, K: int, out: torch.Tensor | None = None,
                         sel: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """Top-K sparse decode: each (sequence, kv head) attends its K blocks
        with the largest score bound plus all fp16 tokens. ``sel``, if given,
        is a CUDA int32 tensor [B*Hkv][min(K, nf)] that receives the blocks
        (nf: the largest block count of any sequence)."""
        shp = (self.B, self.Hq, self.d)
        qp = _dev_ptr(q, shp, "q")
        if out is None:
            out = _new(lambda: torch.empty_like(q), stream, q.get_device())
        sp = None
        if sel is not None:
            nf = max(self.seq_counts(b)[1] for b in range(self.B)) if self.ragged else self.counts()[1]
            kc = min(int(K), nf)
            if (not sel.is_cuda or sel.dtype != torch.int32 or not sel.is_contiguous()
                    or tuple(sel.shape) != (self.B * self.Hkv, kc)):
                raise ValueError(f"sel: expected a contiguous CUDA int32 tensor {(self.B * self.Hkv, kc)}")
            sp = sel.data_ptr()
        _check(load().ott_decode_attn_topk(self._h, qp, _dev_ptr(out, shp, "out"), int(K), sp,
                                           _stream(stream)), "ott_decode_attn_topk")
        return out

    def _lens(self, lens):
        if lens is None:
            return None
        if len(lens) != self.B:
            raise ValueError("lens must hold one length per sequence")
        return (C.c_int * self.B)(*[_int32(x, "lens") for x in lens])

    def chunk_attn(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, lens=None, window: int = 0, sinks: int = 0,
                   out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """Attention of n new tokens per sequence over the cache and, causally, one another (ott_chunk_attn): q fp16
        [B][Hq][n][d], k, v fp16 [B][Hkv][n][d], not yet in the cache; it is not changed. ``lens`` (ragged caches): the
        new tokens of each sequence, at most n; rows behind them are neither read nor written. ``window`` > 0: a query
        sees the last ``window`` tokens up to itself and the sequence's first ``sinks``."""
        n = q.shape[2] if isinstance(q, torch.Tensor) and q.dim() == 4 else -1
        shp, kshp = (self.B, self.Hq, n, self.d), (self.B, self.Hkv, n, self.d)
        ptr = [_dev_ptr(q, shp, "q"), _dev_ptr(k, kshp, "k"), _dev_ptr(v, kshp, "v")]
        if out is None:
            out = _new(lambda: torch.empty_like(q), stream, q.get_device())
        ptr.append(_dev_ptr(out, shp, "out"))
        _same_device(self._dev, q, k, v, out)
        _on_device(self._dev, load().ott_chunk_attn, "ott_chunk_attn", self._h, *ptr, n, self._lens(lens),
                   _int32(window, "window"), _int32(sinks, "sinks"), _stream_of(stream, self._dev))
        return out

    def append_chunk(self, k: torch.Tensor, v: torch.Tensor, lens=None, stream=None):
        """Append n tokens per sequence, k, v fp16 [B][Hkv][n][d] (ott_append_chunk): the same as n appends. ``lens``
        (ragged caches): sequence b takes its first lens[b] tokens, 0 included."""
        n = k.shape[2] if isinstance(k, torch.Tensor) and k.dim() == 4 else -1
        shp = (self.B, self.Hkv, n, self.d)
        ptr = [_dev_ptr(k, shp, "k"), _dev_ptr(v, shp, "v")]
        _same_device(self._dev, k, v)
        _on_device(self._dev, load().ott_append_chunk, "ott_append_chunk", self._h, *ptr, n, self._lens(lens),
                   _stream_of(stream, self._dev))

    def decode_attn_window(self, q: torch.Tensor, window: int, sinks: int = 0, out: torch.Tensor | None = None,
                           stream=None) -> torch.Tensor:
        """decode_attn over the last ``window`` tokens and the first ``sinks`` (ott_decode_attn_window; window 0: all)."""
        shp = (self.B, self.Hq, self.d)
        qp = _dev_ptr(q, shp, "q")
        if out is None:
            out = _new(lambda: torch.empty_like(q), stream, q.get_device())
        op = _dev_ptr(out, shp, "out")
        _same_device(self._dev, q, out)
        _on_device(self._dev, load().ott_decode_attn_window, "ott_decode_attn_window", self._h, qp, op,
                   _int32(window, "window"), _int32(sinks, "sinks"), _stream_of(stream, self._dev))
        return out

    def counts(self):
        T, nf, tail, npool = C.c_longlong(), C.c_int(), C.c_int(), C.c_int()
        _check(load().ott_get_counts(self._h, C.byref(T), C.byref(nf), C.byref(tail), C.byref(npool)),
               "ott_get_counts")
        return T.value, nf.value, tail.value, npool.value

    def seq_counts(self, b: int):
        T, nf, tail, npool = C.c_longlong(), C.c_int(), C.c_int(), C.c_int()
        _check(load().ott_get_seq_counts(self._h, b, C.byref(T), C.byref(nf), C.byref(tail), C.byref(npool)),
               "ott_get_seq_counts")
        return T.value, nf.value, tail.value, npool.value

    def release_seq(self, b: int, stream=None):
        """Sequence b finishes: it drops its tokens (and its pool blocks)."""
        _check(load().ott_release_seq(self._h, int(b), _stream(stream)), "ott_release_seq")

    def prefill_seq(self, b: int, K: torch.Tensor, V: torch.Tensor, stream=None):
        """Fill the empty sequence b with a prompt: K, V fp16 [Hkv][L][d] on the device."""
        L = K.shape[1] if K.dim() == 3 else -1
        shp = (self.Hkv, L, self.d)
        _check(load().ott_prefill_seq(self._h, int(b), _dev_ptr(K, shp, "K"), _dev_ptr(V, shp, "V"), L,
                                      _stream(stream)), "ott_prefill_seq")

    def free_blocks(self) -> int:
        """Free blocks of the paged pool (-1 without one)."""
        return int(load().ott_free_blocks(self._h))

    def cold_sizes(self):
        """Cold-pool policy: (block sizes [U][nf], cold-pool sizes [U]) from the device."""
        import numpy as np
        U, nf = self.B * self.Hkv, self.counts()[1]
        bc = np.zeros((U, max(nf, 1)), np.int32)
        nc = np.zeros(U, np.int32)
        _check(load().ott_export_cold(self._h, 0, U, bc.ctypes.data, nc.ctypes.data, None, None, None),
               "ott_export_cold")
        return bc[:, :nf], nc

    def block_count(self, j: int) -> int:
        rc = load().ott_block_count(self._h, j)
        if rc < 0:
            raise OTTError(rc, "ott_block_count")
        return rc

    def device_bytes(self) -> int:
        return int(load().ott_device_bytes(self._h))

    def check_device(self):
        _check(load().ott_check_device(self._h), "ott_check_device")

    def export_state(self, u0: int = 0, nu: int | None = None) -> dict:
        """Canonical host arrays of units [u0, u0+nu) (numpy). In a ragged
        batch the units must belong to one sequence."""
        import numpy as np
        nu = self.B * self.Hkv - u0 if nu is None else nu
        T, nf, nt, npool = self.seq_counts(u0 // self.Hkv)
        G, P, d = self.G, self.P, self.d
        e = dict(
            bidx=np.zeros((nu, nf, G), np.int32),
            kcode=np.zeros((nu, nf, G, d // 4), np.uint8),
            ks=np.zeros((nu, nf, d), np.uint16), kz=np.zeros((nu, nf, d), np.uint16),
            vcode=np.zeros((nu, nf, G, d // 4), np.uint8),
            vs=np.zeros((nu, nf, G, d // 32), np.uint16), vz=np.zeros((nu, nf, G, d // 32), np.uint16),
            tk=np.zeros((nu, nt, d), np.uint16), tv=np.zeros((nu, nt, d), np.uint16),
            pidx=np.zeros((nu, P), np.int32), pnorm=np.zeros((nu, P), np.uint32),
            pk=np.zeros((nu, P, d), np.uint16), pv=np.zeros((nu, P, d), np.uint16),
        )
        st = StateExport(**{k: (v.ctypes.data if v.size else None) for k, v in e.items()})
        _check(load().ott_export_state(self._h, u0, nu, C.byref(st)), "ott_export_state")
        if self.cold is None:
            e["bcount"] = np.array([self.block_count(j) for j in range(nf)], np.int32)
        else:
            Cc = int(self.cold)
            bc = np.zeros((nu, max(nf, 1)), np.int32)
            nc = np.zeros(nu, np.int32)
            ci = np.zeros((nu, max(Cc, 1)), np.int32)
            ck = np.zeros((nu, max(Cc, 1), d), np.uint16)
            cv = np.zeros((nu, max(Cc, 1), d), np.uint16)
            _check(load().ott_export_cold(self._h, u0, nu, bc.ctypes.data, nc.ctypes.data, ci.ctypes.data,
                                          ck.ctypes.data, cv.ctypes.data), "ott_export_cold")
            e.update(bcount=bc[:, :nf], ncold=nc, cidx=ci[:, :Cc], ck=ck[:, :Cc], cv=cv[:, :Cc])
        e.update(T=T, nf=nf, tail=nt, npool=npool)
        return e


class ByteCache:
    """One cache (one attention layer) held in 8 bits, for layers that 2 bits hurt (``ott_byte_*``): keys and values of
    complete blocks of G tokens (32, 64 or 128) as codes of one byte with one scale for the keys and one for the values
    of each block and kv head, the tokens of the open block in fp16. ``fmt``: "int8" or "e4m3". Every sequence keeps
    its own length. ``pool_blocks``: the complete blocks of all (sequence, kv head) units come from one pool.

    Calls go to the given stream, or to the current one of the cache's device, on which all tensors lie; they are made
    one after another on one stream, or ordered by events."""

    FORMATS = {"int8": 0, "e4m3": 1}

    def __init__(self, B, Hq, Hkv, d, G=64, fmt="int8", max_tokens=8192, pool_blocks=None):
        self._L = L = load()
        if fmt not in self.FORMATS:
            raise ValueError(f"fmt: expected one of {tuple(self.FORMATS)}, got {fmt!r}")
        pool = 0 if pool_blocks is None else _int32(pool_blocks, "pool_blocks")
        if pool_blocks is not None and pool < 1:
            raise ValueError("pool_blocks: at least one block")
        self.B, self.Hq, self.Hkv, self.d, self.G, self.fmt, self.max_tokens = B, Hq, Hkv, d, G, fmt, max_tokens
        self._h = C.c_void_p()
        self._dev = torch.cuda.current_device()
        self._qshape, self._kshape = (B, Hq, d), (B, Hkv, d)
        sizes = [_int32(x, n) for x, n in ((B, "B"), (Hq, "Hq"), (Hkv, "Hkv"), (d, "d"), (G, "G"))]
        _check(L.ott_byte_create(*sizes, self.FORMATS[fmt], _int32(max_tokens, "max_tokens"), pool,
                                 C.byref(self._h)), "ott_byte_create")

    def close(self):
        if getattr(self, "_h", None) and self._h.value:
            load().ott_byte_destroy(self._h)
            self._h = C.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    @property
    def handle(self) -> int:
        return self._h.value

    # (Small calls end on the device before the next one is queued: checks are one expression, and the current stream
    # and device come from the calls that torch's own wrappers make: a decode step's call 15 -> 8 us.)
    def _call(self, fn, what, *args, stream):
        dev = self._dev
        s = _raw_stream(dev) if stream is None else stream.cuda_stream
        if _raw_device() == dev:
            rc = fn(self._h, *args, s)
            if rc:
                _check(rc, what)
        else:
            _on_device(dev, fn, what, self._h, *args, s)

    def _ptr(self, t, shape, name) -> int:
        if isinstance(t, torch.Tensor) and t.dtype is torch.float16 and t.get_device() == self._dev and t.shape == shape \
                and t.is_contiguous():
            return t.data_ptr()
        _dev_ptr(t, shape, name)   # says what is wrong, but for the device
        raise ValueError(f"{name}: on {t.device}, the cache is on cuda:{self._dev}")

    def _lens(self, lens):
        if lens is None:
            return None
        try:
            lens = array.array("i", [*lens])   # (of the list: bytes alone would be taken for the array's memory)
        except OverflowError:
            raise ValueError("lens: a length does not fit 32 bits") from None
        if len(lens) != self.B:   # the library reads B of them
            raise ValueError("lens must hold one length per sequence")
        return lens

    def _append(self, k, v, n, shape, lens, stream):
        lens = self._lens(lens)   # alive during the call
        self._call(self._L.ott_byte_append, "ott_byte_append", self._ptr(k, shape, "k"), self._ptr(v, shape, "v"), n,
                   lens and lens.buffer_info()[0], stream=stream)

    def append(self, k: torch.Tensor, v: torch.Tensor, stream=None):
        """One token to every sequence: k, v fp16 [B][Hkv][d]."""
        self._append(k, v, 1, self._kshape, None, stream)

    def append_chunk(self, k: torch.Tensor, v: torch.Tensor, lens=None, stream=None):
        """n tokens per sequence, k, v fp16 [B][Hkv][n][d] (ott_byte_append); ``lens``: sequence b takes its first lens[b],
        0 included. What the cache holds does not depend on how the tokens are cut into calls."""
        n = k.shape[2] if isinstance(k, torch.Tensor) and k.dim() == 4 else -1
        self._append(k, v, n, (self.B, self.Hkv, n, self.d), lens, stream)

    def prefill(self, K: torch.Tensor, V: torch.Tensor, stream=None):
        """A prompt of L tokens for every sequence of an empty cache: K, V fp16 [B][Hkv][L][d]."""
        self.prefill_lens(K, V, None, stream)

    def prefill_lens(self, K: torch.Tensor, V: torch.Tensor, lens, stream=None):
        """The same with lens[b] tokens for sequence b."""
        if self.seq_counts(-1)[0]:
            raise OTTError(OTT_ERR_STATE, "prefill of a cache that holds tokens")
        self.append_chunk(K, V, lens, stream)

    def prefill_seq(self, b: int, K: torch.Tensor, V: torch.Tensor, stream=None):
        """A prompt for the empty sequence b: K, V fp16 [Hkv][L][d]."""
        if self.seq_counts(b)[0]:
            raise OTTError(OTT_ERR_STATE, "prefill of a sequence that holds tokens")
        n = K.shape[1] if isinstance(K, torch.Tensor) and K.dim() == 3 else -1
        shp = (self.Hkv, n, self.d)
        self._call(self._L.ott_byte_append_seq, "ott_byte_append_seq", _int32(b, "b"), self._ptr(K, shp, "K"),
                   self._ptr(V, shp, "V"), n, stream=stream)

    def read(self, start: int, n: int, out_k: torch.Tensor | None = None, out_v: torch.Tensor | None = None, stream=None):
        """Tokens start .. start + n - 1 of every sequence as the cache holds them (ott_byte_read): keys and values, fp16
        [B][Hkv][n][d]. Rows of tokens that a sequence does not hold stay as they are (zero in a new tensor)."""
        n = _int32(n, "n")
        shp = (self.B, self.Hkv, n, self.d)
        zeros = lambda: torch.zeros(shp, dtype=torch.float16, device=f"cuda:{self._dev}")
        if out_k is None:
            out_k = _new(zeros, stream, self._dev)
        if out_v is None:
            out_v = _new(zeros, stream, self._dev)
        self._call(self._L.ott_byte_read, "ott_byte_read", self._ptr(out_k, shp, "out_k"), self._ptr(out_v, shp, "out_v"),
                   _int32(start, "start"), n, stream=stream)
        return out_k, out_v

    def decode_attn(self, q: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """One query per sequence over all its tokens: q fp16 [B][Hq][d] -> [B][Hq][d]."""
        return self.decode_attn_topk(q, 0, out, None, stream)

    def decode_attn_topk(self, q: torch.Tensor, K: int, out: torch.Tensor | None = None, sel: torch.Tensor | None = None,
                         stream=None) -> torch.Tensor:
        """decode_attn over the K complete blocks with the largest bound of each (sequence, kv head) and the open block
        (ott_byte_decode; K = 0: all). ``sel``: int32 [B][1][Hkv][min(K, most blocks of a sequence)] (or without the
        1), receives the blocks."""
        qp = self._ptr(q, self._qshape, "q")
        if out is None:
            out = _new(lambda: torch.empty_like(q), stream, self._dev)
        self._call(self._L.ott_byte_decode, "ott_byte_decode", qp, self._ptr(out, self._qshape, "out"), _int32(K, "K"),
                   self._sel(sel, 1, K), stream=stream)
        return out

    def chunk_attn(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, lens=None, out: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
        """n new tokens per sequence over the cache and, causally, one another (ott_byte_attn): q fp16 [B][Hq][n][d], k, v
        fp16 [B][Hkv][n][d], not yet in the cache; it is not changed. ``lens``: the new tokens of each sequence; rows
        behind them are neither read nor written."""
        return self.chunk_attn_topk(q, k, v, 0, lens, out, None, stream)

    def chunk_attn_topk(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, K: int, lens=None,
                        out: torch.Tensor | None = None, sel: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """chunk_attn in which every token attends, for each kv head, the K complete blocks with its largest bounds, the
        open block, and new tokens up to itself. ``sel``: int32 [B][n][Hkv][min(K, most blocks of a sequence)], receives
        the blocks."""
        n = q.shape[2] if isinstance(q, torch.Tensor) and q.dim() == 4 else -1
        shp, kshp = (self.B, self.Hq, n, self.d), (self.B, self.Hkv, n, self.d)
        ptr = [self._ptr(q, shp, "q"), self._ptr(k, kshp, "k"), self._ptr(v, kshp, "v")]
        if out is None:
            out = _new(lambda: torch.empty_like(q), stream, self._dev)
        lens = self._lens(lens)
        self._call(self._L.ott_byte_attn, "ott_byte_attn", *ptr, self._ptr(out, shp, "out"), n,
                   lens and lens.buffer_info()[0], _int32(K, "K"), self._sel(sel, n, K), stream=stream)
        return out

    def _sel(self, sel, n, K):
        if sel is None:
            return None
        slots = min(int(K), self.seq_counts(-1)[1])
        shapes = [(self.B, n, self.Hkv, slots)] + ([(self.B, self.Hkv, slots)] if n == 1 else [])
        if not isinstance(sel, torch.Tensor) or not sel.is_cuda or sel.dtype != torch.int32:
            raise TypeError("sel: expected a CUDA int32 tensor")
        if tuple(sel.shape) not in shapes or not sel.is_contiguous() or sel.get_device() != self._dev:
            raise ValueError(f"sel: expected contiguous shape {shapes[0]} on cuda:{self._dev}, got {tuple(sel.shape)}")
        return sel.data_ptr()

    def release_seq(self, b: int, stream=None):
        """Sequence b drops its tokens (and its pool blocks)."""
        self._call(self._L.ott_byte_release, "ott_byte_release", _int32(b, "b"), stream=stream)

    def reset(self, stream=None):
        """Every sequence drops its tokens."""
        self._call(self._L.ott_byte_reset, "ott_byte_reset", stream=stream)

    def seq_counts(self, b: int):
        """(tokens of sequence b, its complete blocks per kv head); b = -1: of the longest sequence."""
        T, nb = C.c_longlong(), C.c_int()
        _check(self._L.ott_byte_counts(self._h, _int32(b, "b"), C.byref(T), C.byref(nb)), "ott_byte_counts")
        return T.value, nb.value

    def free_blocks(self) -> int:
        """Free blocks of the pool (-1 without one)."""
        return int(self._L.ott_byte_free_blocks(self._h))

    def device_bytes(self) -> int:
        return int(self._L.ott_byte_bytes(self._h))

    def check_device(self):
        _on_device(self._dev, self._L.ott_byte_check, "ott_byte_check", self._h)
