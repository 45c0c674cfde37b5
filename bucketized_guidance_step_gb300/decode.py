"""Python binding of the decode operators (``include/gs_decode.h``): argument marshalling only.

A ``PagedCache`` describes a key-value cache in the caller's tensors; its methods are the
calls on it. ``guided_logits`` turns a step's logits into the next tokens. Every call has a
``prepare_*`` form that checks the arguments once and returns a ``Call``: calling it launches
the same work again on the same buffers (their contents may change, their addresses may not),
on their device and its ``torch.cuda.current_stream()``, as a sampler's loop or a CUDA graph's
capture does.

As in ``gs``, the arithmetic is the library's; a missing library raises ``GSLibraryError``.
"""

from __future__ import annotations

import ctypes
import threading
from typing import Optional

from . import gs
from .gs import GSError, _dtype_code

# ---- constants mirrored from include/gs_decode.h -------------------------------
GS_DEV_NO_PAGE, GS_DEV_BAD_SEQ, GS_DEV_EMPTY_ROW = 16, 32, 64
GS_MAX_SEQS = 8192
GS_CHUNK_COUNTERS = 1024

EXPORTS = ("gs_pages_workspace", "gs_pages_extend", "gs_pages_fork", "gs_pages_free",
           "gs_pages_compact", "gs_kv_write", "gs_paged_attention_workspace",
           "gs_paged_attention", "gs_chunk_attention_workspace", "gs_chunk_attention",
           "gs_guided_logits_workspace", "gs_guided_logits", "gs_sample",
           "gs_decode_status_from_word")

_I32, _I64, _P, _F = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float


class KVCacheDesc(ctypes.Structure):
    _fields_ = [("dtype", _I32), ("layers", _I32), ("pages", _I32), ("kv_heads", _I32),
                ("page", _I32), ("dim", _I32), ("k", _P), ("v", _P), ("layer_stride", _I64),
                ("page_stride", _I64), ("head_stride", _I64), ("token_stride", _I64),
                ("seqs", _I32), ("cols", _I32), ("table", _P), ("lens", _P), ("refs", _P),
                ("dev_status", _P), ("workspace", _P), ("workspace_bytes", _I64)]


class PagedAttentionArgs(ctypes.Structure):
    _fields_ = [("cache", ctypes.POINTER(KVCacheDesc)), ("layer", _I32), ("batch", _I32),
                ("seq", _P), ("q_heads", _I32), ("q", _P), ("q_batch_stride", _I64),
                ("q_head_stride", _I64), ("k_new", _P), ("v_new", _P),
                ("new_batch_stride", _I64), ("new_head_stride", _I64), ("scale", _F),
                ("window", _I32), ("sinks", _I32), ("out", _P), ("out_batch_stride", _I64),
                ("out_head_stride", _I64), ("lse", _P), ("workspace", _P),
                ("workspace_bytes", _I64)]


class ChunkAttentionArgs(ctypes.Structure):
    _fields_ = [("cache", ctypes.POINTER(KVCacheDesc)), ("layer", _I32), ("tokens", _I32),
                ("n", _I32), ("seq", _P), ("start", _P), ("q_heads", _I32), ("q", _P),
                ("q_token_stride", _I64), ("q_head_stride", _I64), ("scale", _F),
                ("window", _I32), ("sinks", _I32), ("split_weights", _I32), ("out", _P),
                ("out_token_stride", _I64),
                ("out_head_stride", _I64), ("lse", _P), ("workspace", _P),
                ("workspace_bytes", _I64)]


class GuidedLogitsArgs(ctypes.Structure):
    _fields_ = [("batch", _I32), ("vocab", _I32), ("dtype", _I32), ("uncond", _P), ("cond", _P),
                ("row_stride", _I64), ("step_idx", _P), ("step", _I32), ("scale_lut", _P),
                ("n_lut", _I32), ("cfg", _F), ("bias", _P), ("bias_stride", _I64),
                ("tokens", _P), ("tokens_stride", _I64), ("tokens_len", _P), ("prompt_len", _P),
                ("repetition", _P), ("frequency", _P), ("presence", _P), ("temperature", _P),
                ("mask", _P), ("mask_stride", _I64), ("mask_present", _P), ("noise", _P),
                ("noise_stride", _I64), ("out", _P), ("out_stride", _I64), ("token", _P),
                ("logprob", _P), ("dev_status", _P), ("workspace", _P),
                ("workspace_bytes", _I64)]


class SampleArgs(ctypes.Structure):
    _fields_ = [("batch", _I32), ("vocab", _I32), ("dtype", _I32), ("logits", _P),
                ("row_stride", _I64), ("temperature", _P), ("top_k", _P), ("top_p", _P),
                ("min_p", _P), ("noise", _P), ("noise_stride", _I64), ("token", _P),
                ("logprob", _P), ("dev_status", _P)]


_ready = False
_lock = threading.Lock()


def load() -> ctypes.CDLL:
    """libgs.so with the decode entry points' argument types set."""
    global _ready
    lib = gs.load()
    if _ready:
        return lib
    with _lock:
        cache = ctypes.POINTER(KVCacheDesc)
        lib.gs_pages_workspace.argtypes = [cache, _P]
        lib.gs_pages_extend.argtypes = [cache, _P, _P, _I32, _P]
        lib.gs_pages_fork.argtypes = [cache, _P, _P, _I32, _P]
        lib.gs_pages_free.argtypes = [cache, _P, _I32, _P]
        lib.gs_pages_compact.argtypes = [cache, _P, _P, _P, _P]
        lib.gs_kv_write.argtypes = [cache, _I32, _P, _P, _I64, _I64, _I32, _P, _P, _I32, _P]
        lib.gs_paged_attention_workspace.argtypes = [ctypes.POINTER(PagedAttentionArgs), _P]
        lib.gs_paged_attention.argtypes = [ctypes.POINTER(PagedAttentionArgs), _P]
        lib.gs_chunk_attention_workspace.argtypes = [ctypes.POINTER(ChunkAttentionArgs), _P]
        lib.gs_chunk_attention.argtypes = [ctypes.POINTER(ChunkAttentionArgs), _P]
        lib.gs_guided_logits_workspace.argtypes = [ctypes.POINTER(GuidedLogitsArgs), _P]
        lib.gs_guided_logits.argtypes = [ctypes.POINTER(GuidedLogitsArgs), _P]
        lib.gs_sample.argtypes = [ctypes.POINTER(SampleArgs), _P]
        lib.gs_decode_status_from_word.argtypes = [ctypes.c_uint32]
        for f in EXPORTS:
            getattr(lib, f).restype = _I32
        _ready = True
    return lib


def status_from_word(word: int) -> int:
    """gs_decode_status_from_word: the status of a device status word of these calls."""
    return int(load().gs_decode_status_from_word(int(word) & 0xFFFFFFFF))


class Call:
    """A checked call on fixed buffers: ``call()`` launches it on the current stream.

    The call keeps its tensors and its workspace alive; keep the call until its work is done
    where that runs on another stream than the tensors were made on, or in a captured graph.
    A workspace serves one call at a time: two calls of attention or logits in flight at once need
    a ``Call`` each, and calls on one cache's pages, whose workspace is the cache's, are ordered
    by the caller whatever their ``Call`` objects."""

    def __init__(self, name: str, args, device, keep):
        import torch
        self._name = name
        self._fn = getattr(load(), name)
        self._args = args                       # ctypes values, the stream excepted
        self._keep = keep                       # tensors and structs behind the pointers
        self._device = device.index
        # The library launches on the current device: a stream's handle does not name one (the
        # default stream's is 0 on each).
        self._current = torch._C._cuda_getDevice
        self._guard = torch.cuda.device
        # The handle alone: torch.cuda.current_stream() builds a Stream object around it (1 us).
        self._stream = torch._C._cuda_getCurrentRawStream

    def __call__(self) -> None:
        if self._current() == self._device:
            status = self._fn(*self._args, self._stream(self._device))
        else:
            with self._guard(self._device):
                status = self._fn(*self._args, self._stream(self._device))
        if status != gs.GS_OK:
            raise GSError(self._name, status)


def _ptr(t, name: str, device, dtype=None, shape=None, contiguous: bool = True) -> Optional[int]:
    """The data pointer of a tensor after its checks; None stays None."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _stride(t, dim: int) -> int:
    """The stride of a dimension; 0 where it has one entry (it is never stepped)."""
    return t.stride(dim) if t.shape[dim] > 1 else 0


def _last_dense(t, name: str) -> None:
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}'s last dimension must be dense")


def _no_overlap(t, name: str) -> None:
    """A written tensor's elements are all its own."""
    need = 1
    for stride, size in sorted((t.stride(i), t.shape[i]) for i in range(t.dim()) if t.shape[i] > 1):
        if stride < need:
            raise ValueError(f"{name}'s elements overlap")
        need = stride * (size - 1) + need


class PagedCache:
    """A paged key-value cache in the caller's tensors (see gs_kv_cache).

    k, v: [layers, pages, kv_heads, page, dim], fp32, bf16 or fp16, the same strides (any
    order of the first four dimensions: a permuted view serves), the last dimension dense,
    every row on 16 bytes. table: int32 [seqs, cols], lens: int32 [seqs], refs: int32 [pages]
    (lens and refs start as zeros). status: int32 [1], device flags OR-ed in. workspace: int32,
    made (zeros) where none is given; caches over one table (k and v of a layer each, say) pass the
    first one's .workspace, as it also keeps which sequences the last extension refused.
    """

    def __init__(self, k, v, table, lens, refs, *, status=None, workspace=None):
        import torch
        if k.dim() != 5 or tuple(k.shape) != tuple(v.shape) or k.dtype != v.dtype:
            raise ValueError("k and v must be [layers, pages, kv_heads, page, dim] alike")
        if any(k.shape[i] > 1 and k.stride(i) != v.stride(i) for i in range(5)):
            raise ValueError("k and v must have the same strides")
        if table.dim() != 2:
            raise ValueError("table must be [seqs, cols]")
        dev = k.device
        lib = load()
        for name, t in (("k", k), ("v", v)):
            _last_dense(t, name)
            _no_overlap(t, name)
        d = KVCacheDesc()
        d.dtype = _dtype_code(k)
        d.layers, d.pages, d.kv_heads, d.page, d.dim = k.shape
        d.k, d.v = _ptr(k, "k", dev, contiguous=False), _ptr(v, "v", dev, contiguous=False)
        d.layer_stride, d.page_stride, d.head_stride, d.token_stride = (_stride(k, i) for i in range(4))
        d.seqs, d.cols = table.shape
        d.table = _ptr(table, "table", dev, torch.int32)
        d.lens = _ptr(lens, "lens", dev, torch.int32, (d.seqs,))
        d.refs = _ptr(refs, "refs", dev, torch.int32, (d.pages,))
        d.dev_status = _ptr(status, "status", dev, torch.int32)
        n = ctypes.c_int64(0)
        gs._check("gs_pages_workspace", lib.gs_pages_workspace(ctypes.byref(d), ctypes.byref(n)))
        if workspace is None:
            workspace = torch.zeros((n.value + 3) // 4, dtype=torch.int32, device=dev)
        elif workspace.numel() * 4 < n.value:
            raise ValueError(f"workspace must hold {(n.value + 3) // 4} words")
        d.workspace, d.workspace_bytes = _ptr(workspace, "workspace", dev, torch.int32), workspace.numel() * 4
        self.k, self.v, self.table, self.lens, self.refs, self.status = k, v, table, lens, refs, status
        self.workspace = workspace
        self.device = dev
        self._desc = d
        self._keep = (k, v, table, lens, refs, status, workspace)

    def _call(self, name, args, *keep) -> Call:
        return Call(name, (ctypes.byref(self._desc),) + args, self.device, (self, self._desc) + keep)

    def _list(self, t, name: str, n: Optional[int] = None):
        import torch
        if t is not None and t.dim() != 1:
            raise ValueError(f"{name} must be one-dimensional")
        return _ptr(t, name, self.device, torch.int32, None if n is None else (n,))

    def prepare_extend(self, seq, add=None) -> Call:
        n = seq.numel()
        return self._call("gs_pages_extend", (self._list(seq, "seq"), self._list(add, "add", n), n), seq, add)

    def extend(self, seq, add=None) -> None:
        """gs_pages_extend: room for add[i] (default 1) more tokens of sequence seq[i]."""
        self.prepare_extend(seq, add)()

    def prepare_fork(self, src, dst) -> Call:
        n = src.numel()
        return self._call("gs_pages_fork", (self._list(src, "src"), self._list(dst, "dst", n), n), src, dst)

    def fork(self, src, dst) -> None:
        """gs_pages_fork: sequence dst[i] becomes a copy of src[i] that shares its full pages."""
        self.prepare_fork(src, dst)()

    def prepare_free(self, seq) -> Call:
        return self._call("gs_pages_free", (self._list(seq, "seq"), seq.numel()), seq)

    def free(self, seq) -> None:
        """gs_pages_free: the listed sequences release their pages."""
        self.prepare_free(seq)()

    def prepare_compact(self, *, table_out=None, refs_out=None, live=None) -> Call:
        import torch
        d = self._desc
        table_out = self.table if table_out is None else table_out
        refs_out = self.refs if refs_out is None else refs_out
        return self._call("gs_pages_compact",
                          (_ptr(table_out, "table_out", self.device, torch.int32, (d.seqs, d.cols)),
                           _ptr(refs_out, "refs_out", self.device, torch.int32, (d.pages,)),
                           _ptr(live, "live", self.device, torch.int32, (1,))), table_out, refs_out, live)

    def compact(self, *, table_out=None, refs_out=None, live=None) -> None:
        """gs_pages_compact: the held pages move to the front of the pool (k and v in place;
        table and refs in place unless table_out and refs_out are given)."""
        self.prepare_compact(table_out=table_out, refs_out=refs_out, live=live)()

    def prepare_write(self, layer: int, k, v, seq, start) -> Call:
        d = self._desc
        if k.dim() != 3 or tuple(k.shape) != tuple(v.shape) or tuple(k.shape[1:]) != (d.kv_heads, d.dim):
            raise ValueError(f"k and v must be [tokens, {d.kv_heads}, {d.dim}]")
        if any(k.shape[i] > 1 and k.stride(i) != v.stride(i) for i in range(3)):
            raise ValueError("k and v must have the same strides")
        _last_dense(k, "k")
        n = seq.numel()
        return self._call("gs_kv_write",
                          (int(layer), _ptr(k, "k", self.device, self.k.dtype, contiguous=False),
                           _ptr(v, "v", self.device, self.k.dtype, contiguous=False),
                           _stride(k, 0), _stride(k, 1), k.shape[0], self._list(seq, "seq"),
                           self._list(start, "start", n + 1), n), k, v, seq, start)

    def write(self, layer: int, k, v, seq, start) -> None:
        """gs_kv_write: rows start[i] .. start[i+1]-1 of k and v ([tokens, kv_heads, dim]) are
        the last tokens of sequence seq[i] in this layer."""
        self.prepare_write(layer, k, v, seq, start)()

    def prepare_attention(self, q, layer: int, *, seq=None, k_new=None, v_new=None,
                          scale: Optional[float] = None, window: int = 0, sinks: int = 0,
                          out=None, lse=None) -> Call:
        import torch
        d, dev, dt = self._desc, self.device, self.k.dtype
        if q.dim() != 3 or q.shape[2] != d.dim:
            raise ValueError(f"q must be [batch, q_heads, {d.dim}]")
        B, Hq, D = q.shape
        if out is None or tuple(out.shape) != tuple(q.shape):
            raise ValueError("out must have the shape of q")
        if (k_new is None) != (v_new is None):
            raise ValueError("pass both k_new and v_new, or neither")
        a = PagedAttentionArgs()
        a.cache = ctypes.pointer(d)
        a.layer, a.batch, a.q_heads = int(layer), B, Hq
        a.seq = self._list(seq, "seq", B)
        for name, t in (("q", q), ("out", out)):
            _last_dense(t, name)
        _no_overlap(out, "out")
        a.q, a.out = _ptr(q, "q", dev, dt, contiguous=False), _ptr(out, "out", dev, dt, contiguous=False)
        a.q_batch_stride, a.q_head_stride = _stride(q, 0), _stride(q, 1)
        a.out_batch_stride, a.out_head_stride = _stride(out, 0), _stride(out, 1)
        if k_new is not None:
            for name, t in (("k_new", k_new), ("v_new", v_new)):
                if tuple(t.shape) != (B, d.kv_heads, D):
                    raise ValueError(f"{name} must be [{B}, {d.kv_heads}, {D}]")
                _last_dense(t, name)
            if any(k_new.shape[i] > 1 and k_new.stride(i) != v_new.stride(i) for i in range(2)):
                raise ValueError("k_new and v_new must have the same strides")
            a.k_new = _ptr(k_new, "k_new", dev, dt, contiguous=False)
            a.v_new = _ptr(v_new, "v_new", dev, dt, contiguous=False)
            a.new_batch_stride, a.new_head_stride = _stride(k_new, 0), _stride(k_new, 1)
        a.scale = float(D) ** -0.5 if scale is None else float(scale)
        a.window, a.sinks = int(window), int(sinks)
        a.lse = _ptr(lse, "lse", dev, torch.float32, (B, Hq))
        work = _zeroed("gs_paged_attention_workspace", a, dev, B * Hq)
        return Call("gs_paged_attention", (ctypes.byref(a),), dev,
                    (self, d, a, q, out, lse, seq, k_new, v_new, work))

    def attention(self, q, layer: int, *, out=None, **kw):
        """gs_paged_attention: q [batch, q_heads, dim] over the cache's layer; returns out.

        seq: int32 [batch] (default: row b reads sequence b); k_new, v_new: [batch, kv_heads,
        dim], stored at each sequence's last position first; scale (default dim ** -0.5);
        window and sinks: only the last `window` and the first `sinks` positions; lse: fp32
        [batch, q_heads], receives the log-sum-exp of the scaled scores."""
        import torch
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        self.prepare_attention(q, layer, out=out, **kw)()
        return out

    def prepare_chunk_attention(self, q, layer: int, seq, start, *, scale: Optional[float] = None,
                                window: int = 0, sinks: int = 0, split_weights: bool = False,
                                out=None, lse=None) -> Call:
        import torch
        d, dev, dt = self._desc, self.device, self.k.dtype
        if q.dim() != 3 or q.shape[2] != d.dim:
            raise ValueError(f"q must be [tokens, q_heads, {d.dim}]")
        T, Hq, D = q.shape
        if out is None or tuple(out.shape) != tuple(q.shape):
            raise ValueError("out must have the shape of q")
        a = ChunkAttentionArgs()
        a.cache = ctypes.pointer(d)
        a.layer, a.tokens, a.q_heads, a.n = int(layer), T, Hq, seq.numel()
        a.seq, a.start = self._list(seq, "seq"), self._list(start, "start", a.n + 1)
        for name, t in (("q", q), ("out", out)):
            _last_dense(t, name)
        _no_overlap(out, "out")
        a.q, a.out = _ptr(q, "q", dev, dt, contiguous=False), _ptr(out, "out", dev, dt, contiguous=False)
        a.q_token_stride, a.q_head_stride = _stride(q, 0), _stride(q, 1)
        a.out_token_stride, a.out_head_stride = _stride(out, 0), _stride(out, 1)
        a.scale = float(D) ** -0.5 if scale is None else float(scale)
        a.window, a.sinks, a.split_weights = int(window), int(sinks), int(split_weights)
        a.lse = _ptr(lse, "lse", dev, torch.float32, (T, Hq))
        work = _zeroed("gs_chunk_attention_workspace", a, dev, GS_CHUNK_COUNTERS)
        return Call("gs_chunk_attention", (ctypes.byref(a),), dev, (self, d, a, q, out, lse, seq, start, work))

    def chunk_attention(self, q, layer: int, seq, start, *, out=None, **kw):
        """gs_chunk_attention: rows start[i] .. start[i+1]-1 of q [tokens, q_heads, dim] are the last
        tokens of sequence seq[i], whose K and V the cache's layer holds; each attends over the
        positions up to its own. Returns out.

        seq: int32 [n], start: int32 [n + 1]; scale (default dim ** -0.5); window and sinks: only the
        last `window` positions up to the row's own and the first `sinks`; split_weights: in 16-bit
        caches the softmax's weights enter the product with V as sums of two 16-bit numbers, as in
        attention (up to a quarter more time), else rounded to one; lse: fp32 [tokens, q_heads],
        receives the log-sum-exp of the scaled scores. Rows of no entry are left as they were (zeros,
        where out is made here)."""
        import torch
        if out is None:
            out = torch.zeros(q.shape, dtype=q.dtype, device=q.device)
        self.prepare_chunk_attention(q, layer, seq, start, out=out, **kw)()
        return out


def _zeroed(fn: str, args, device, words: Optional[int] = None):
    """The workspace that `fn` asks for, its first `words` zeroed (None: all), entered into args."""
    import torch
    n = ctypes.c_int64(0)
    with torch.cuda.device(device):
        gs._check(fn, getattr(load(), fn)(ctypes.byref(args), ctypes.byref(n)))
    work = torch.empty(max(1, (n.value + 3) // 4), dtype=torch.int32, device=device)
    work[:words].zero_()
    args.workspace, args.workspace_bytes = work.data_ptr(), work.numel() * 4
    return work


def prepare_guided_logits(logits=None, *, uncond=None, cond=None, stacked=None, step_idx=None,
                          step: int = 0, scale_lut=None, cfg: float = 1.0, bias=None,
                          tokens=None, tokens_len=None, prompt_len=None, repetition=None,
                          frequency=None, presence=None, temperature=None, mask=None,
                          mask_present=None, noise=None, out=None, token=None, logprob=None,
                          status=None) -> Call:
    import torch
    if sum(x is not None for x in (logits, cond, stacked)) != 1:
        raise ValueError("pass one of logits, cond (with uncond) and stacked")
    if stacked is not None:
        if stacked.dim() != 2 or stacked.shape[0] % 2:
            raise ValueError("stacked must be [2B, vocab]")
        half = stacked.shape[0] // 2
        uncond, cond = stacked[:half], stacked[half:]
    elif logits is not None:
        if uncond is not None:
            raise ValueError("uncond goes with cond")
        cond = logits
    if cond.dim() != 2:
        raise ValueError("logits must be [batch, vocab]")
    B, V = cond.shape
    dev = cond.device
    a = GuidedLogitsArgs()
    a.batch, a.vocab, a.dtype = B, V, _dtype_code(cond)
    for name, t in (("uncond", uncond), ("cond", cond)):
        if t is None:
            continue
        if tuple(t.shape) != (B, V) or t.dtype != cond.dtype:
            raise ValueError(f"{name} must be [{B}, {V}] of {cond.dtype}")
        _last_dense(t, name)
    if uncond is not None and _stride(uncond, 0) != _stride(cond, 0):
        raise ValueError("uncond and cond must have the same strides")
    if _stride(cond, 0) < V and B > 1:
        raise ValueError("the rows of the logits overlap")
    a.uncond = _ptr(uncond, "uncond", dev, contiguous=False)
    a.cond = _ptr(cond, "cond", dev, contiguous=False)
    a.row_stride = _stride(cond, 0)
    a.step_idx, a.step = _ptr(step_idx, "step_idx", dev, torch.int32, (B,)), int(step)
    a.scale_lut = _ptr(scale_lut, "scale_lut", dev, torch.float32)
    a.n_lut = 0 if scale_lut is None else scale_lut.numel()
    a.cfg = float(cfg)
    f32, i32 = torch.float32, torch.int32

    def rows(t, name, dtype, width):
        """A [1 or B, width] tensor: its pointer and the stride between its rows."""
        if t is None:
            return None, 0
        if t.dim() != 2 or t.shape[0] not in (1, B) or t.shape[1] != width:
            raise ValueError(f"{name} must be [1 or {B}, {width}]")
        _last_dense(t, name)
        return _ptr(t, name, dev, dtype, contiguous=False), _stride(t, 0)

    a.bias, a.bias_stride = rows(bias, "bias", f32, V)
    a.mask, a.mask_stride = rows(mask, "mask", i32, (V + 31) // 32)
    a.noise, a.noise_stride = rows(noise, "noise", f32, V)
    a.mask_present = _ptr(mask_present, "mask_present", dev, torch.uint8, (B,))
    if tokens is not None:
        if tokens.dim() != 2 or tokens.shape[0] != B:
            raise ValueError(f"tokens must be [{B}, length]")
        if tokens_len is None:
            raise ValueError("tokens needs tokens_len")
        a.tokens, a.tokens_stride = _ptr(tokens, "tokens", dev, i32), tokens.shape[1]
    a.tokens_len = _ptr(tokens_len, "tokens_len", dev, i32, (B,))
    a.prompt_len = _ptr(prompt_len, "prompt_len", dev, i32, (B,))
    a.repetition = _ptr(repetition, "repetition", dev, f32, (B,))
    a.frequency = _ptr(frequency, "frequency", dev, f32, (B,))
    a.presence = _ptr(presence, "presence", dev, f32, (B,))
    a.temperature = _ptr(temperature, "temperature", dev, f32, (B,))
    if out is not None:
        if tuple(out.shape) != (B, V):
            raise ValueError(f"out must be [{B}, {V}]")
        _last_dense(out, "out")
        _no_overlap(out, "out")
        a.out, a.out_stride = _ptr(out, "out", dev, f32, contiguous=False), _stride(out, 0)
    a.token = _ptr(token, "token", dev, i32, (B,))
    a.logprob = _ptr(logprob, "logprob", dev, f32, (B,))
    if out is None and token is None and logprob is None:
        raise ValueError("pass out, token or logprob")
    a.dev_status = _ptr(status, "status", dev, i32)
    work = _zeroed("gs_guided_logits_workspace", a, dev, B)
    return Call("gs_guided_logits", (ctypes.byref(a),), dev,
                (a, uncond, cond, step_idx, scale_lut, bias, tokens, tokens_len, prompt_len,
                 repetition, frequency, presence, temperature, mask, mask_present, noise, out,
                 token, logprob, status, work))


def guided_logits(logits=None, **kw):
    """gs_guided_logits: the final logits and the next tokens; returns (out, token, logprob).

    logits: [B, V], or cond= with uncond=, or stacked= [2B, V] ([uncond; cond]). Scale: cfg, or
    scale_lut (fp32) at step or step_idx (int32 [B]). bias: fp32 [1 or B, V]. History: tokens
    (int32 [B, T]), tokens_len and prompt_len (int32 [B]), with repetition, frequency and
    presence (fp32 [B]). temperature: fp32 [B], <= 0 greedy. mask: int32 [1 or B, ceil(V/32)]
    bit words (1 = allowed), mask_present: uint8 [B]. noise: fp32 [1 or B, V], added where the
    token is chosen. out: fp32 [B, V], token: int32 [B], logprob: fp32 [B] (made if none of
    the three is given). status: int32 [1]."""
    import torch
    if all(kw.get(x) is None for x in ("out", "token", "logprob")):
        src = next(x for x in (logits, kw.get("cond"), kw.get("stacked")) if x is not None)
        B = src.shape[0] // (2 if kw.get("stacked") is not None else 1)
        kw["out"] = torch.empty((B, src.shape[1]), dtype=torch.float32, device=src.device)
        kw["token"] = torch.empty(B, dtype=torch.int32, device=src.device)
        kw["logprob"] = torch.empty(B, dtype=torch.float32, device=src.device)
    prepare_guided_logits(logits, **kw)()
    return kw.get("out"), kw.get("token"), kw.get("logprob")


def prepare_sample(logits, *, temperature=None, top_k=None, top_p=None, min_p=None, noise=None,
                   token=None, logprob=None, status=None) -> Call:
    import torch
    if logits.dim() != 2:
        raise ValueError("logits must be [batch, vocab]")
    B, V = logits.shape
    dev, f32, i32 = logits.device, torch.float32, torch.int32
    a = SampleArgs()
    a.batch, a.vocab, a.dtype = B, V, _dtype_code(logits)
    _last_dense(logits, "logits")
    if _stride(logits, 0) < V and B > 1:
        raise ValueError("the rows of the logits overlap")
    a.logits, a.row_stride = _ptr(logits, "logits", dev, contiguous=False), _stride(logits, 0)
    a.temperature = _ptr(temperature, "temperature", dev, f32, (B,))
    a.top_k = _ptr(top_k, "top_k", dev, i32, (B,))
    a.top_p = _ptr(top_p, "top_p", dev, f32, (B,))
    a.min_p = _ptr(min_p, "min_p", dev, f32, (B,))
    if noise is not None:
        if noise.dim() != 2 or noise.shape[0] not in (1, B) or noise.shape[1] != V:
            raise ValueError(f"noise must be [1 or {B}, {V}]")
        _last_dense(noise, "noise")
        a.noise, a.noise_stride = _ptr(noise, "noise", dev, f32, contiguous=False), _stride(noise, 0)
    if token is None and logprob is None:
        raise ValueError("pass token or logprob")
    a.token = _ptr(token, "token", dev, i32, (B,))
    a.logprob = _ptr(logprob, "logprob", dev, f32, (B,))
    a.dev_status = _ptr(status, "status", dev, i32)
    return Call("gs_sample", (ctypes.byref(a),), dev,
                (a, logits, temperature, top_k, top_p, min_p, noise, token, logprob, status))


def sample(logits, **kw):
    """gs_sample: the next tokens from a step's logits and given random numbers; returns (token, logprob).

    logits: [B, V], fp32, bf16 or fp16 (the z of guided_logits serves). temperature (<= 0 greedy),
    top_p and min_p: fp32 [B], top_k: int32 [B]; tokens are kept by top_k, then top_p of what that left,
    then min_p. noise: fp32 [1 or B, V], added where the token is chosen (Gumbel noise draws from what is
    kept). token: int32 [B], logprob: fp32 [B] (both made if neither is given). status: int32 [1]."""
    import torch
    if kw.get("token") is None and kw.get("logprob") is None:
        kw["token"] = torch.empty(logits.shape[0], dtype=torch.int32, device=logits.device)
        kw["logprob"] = torch.empty(logits.shape[0], dtype=torch.float32, device=logits.device)
    prepare_sample(logits, **kw)()
    return kw.get("token"), kw.get("logprob")
