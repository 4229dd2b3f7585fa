"""Rotary positions and the 8-bit block cache: write, attention, accumulated
attention weights and eviction (include/dllm_rotary.h, include/dllm_cache.h).

Streams.  An object made with a stream queues on it; without one, each call
queues on the stream that is current for the cache's device.  What a call
allocates (outputs that are not given, workspaces) belongs to the stream it
runs on, and tensors passed to a call on another stream than the current
one are kept alive until that stream is done with them.  Ordering between
streams is the caller's.

Objects of another device than a GPU take their checks, but run nothing: a
valid call raises DLLM_ERR_UNSUPPORTED.
"""
from __future__ import annotations

import ctypes as C
import math

import torch

from . import _abi
from ._abi import DLLM_ERR_INVALID_ARG, DLLM_ERR_UNSUPPORTED, DLLM_OK, DllmError

# The current stream's handle: without the Stream object, a fifth of a small call's time.
_stream_handle = torch._C._cuda_getCurrentRawStream

_BF16 = (torch.bfloat16, torch.int16, torch.uint16)   # bf16 data or its bit pattern
_BLOCK = _abi.DLLM_CACHE_BLOCK


def _need(t, name: str, dtypes, shape, device):
    """A contiguous tensor of the documented type, shape and device: the
    kernels read and write exactly these extents."""
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} is not one of {', '.join(map(str, dtypes))}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")


def _heads(t, name: str, heads, dim, device):
    """[T, heads, dim] bf16 of any strides whose last dimension is dense."""
    if t.dtype not in _BF16:
        raise TypeError(f"{name}: dtype {t.dtype} is not bfloat16 or its bit pattern")
    if t.dim() != 3 or (heads is not None and t.shape[1] != heads) or (dim is not None and t.shape[2] != dim):
        want = ["T", "heads" if heads is None else heads, "dim" if dim is None else dim]
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected [{', '.join(map(str, want))}]")
    if t.shape[2] > 1 and t.stride(2) != 1:
        raise ValueError(f"{name}: the last dimension must be dense")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")


def _overlap(x, y) -> bool:
    """Whether heads x [T, H, dim] of any strides share memory with contiguous y."""
    T, H, D = x.shape
    size, delta = x.element_size(), y.data_ptr() - x.data_ptr()
    token, head = x.stride(0) * size if T > 1 else 0, x.stride(1) * size if H > 1 else 0
    # a head shares some if it begins in lo + 1 .. hi - 1, counted from x's first
    lo, hi = delta - D * size, delta + y.numel() * y.element_size()
    if hi <= 0 or lo >= (T - 1) * token + (H - 1) * head or T * H == 0:
        return False
    for begin in range(0, H * head, head) if head else (0,):
        first = max((lo - begin) // token + 1, 0) if token else 0      # the first token behind lo
        if first < T and lo < begin + first * token < hi:
            return True
    return False


class _Queued:
    """Runs library calls on the object's stream, or the current one."""

    def _call(self, where: str, tensors, make):
        """``make(stream)`` queues the call and returns its status."""
        dev = self.device
        if dev.type != "cuda":
            # a GPU, where there is one, would take these pointers for its own
            raise DllmError(DLLM_ERR_UNSUPPORTED, f"{where} on {dev}")
        if self.stream is None and torch.cuda.current_device() == dev.index:
            st = make(_stream_handle(dev.index))
        else:
            with torch.cuda.device(dev):
                stream = self.stream if self.stream is not None else torch.cuda.current_stream(dev)
                if stream != torch.cuda.current_stream(dev):
                    with torch.cuda.stream(stream):
                        st = make(stream.cuda_stream)
                    for t in tensors:
                        if t is not None:
                            t.record_stream(stream)
                else:
                    st = make(stream.cuda_stream)
        if st != DLLM_OK:
            raise DllmError(st, where)


def _device(device) -> torch.device:
    dev = torch.device(device)
    if dev.type == "cuda" and dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    return dev


def _stream(stream, device):
    """The stream an object queues on: one of its device's, or None."""
    if stream is not None and stream.device != device:
        raise ValueError(f"stream: on {stream.device}, expected {device}")
    return stream


class Rotary(_Queued):
    """Rotary positions of heads whose first ``rotary_dim`` dimensions
    (default: all of ``head_dim``) are rotated.

    ``layout``: "half" pairs dimension i with i + rotary_dim / 2,
    "interleaved" 2 i with 2 i + 1.  ``scaling`` for contexts longer than the
    trained one by ``factor``: "none", "linear", "base" or "ramp" (the last
    also takes ``original_len``, ``fast`` and ``slow``); include/dllm_rotary.h
    gives the formulas.  ``magnitude`` stretches the rotated dimensions; None
    means 1, or 0.1 ln(factor) + 1 for "ramp"."""

    def __init__(self, head_dim: int, rotary_dim: int | None = None, base: float = 10000.0, layout: str = "half",
                 scaling: str = "none", factor: float = 1.0, original_len: int = 0, fast: float = 32.0,
                 slow: float = 1.0, magnitude: float | None = None, device="cuda", stream=None):
        if layout not in _abi.ROTARY_LAYOUTS:
            raise ValueError(f"layout {layout!r} is not one of {', '.join(_abi.ROTARY_LAYOUTS)}")
        if scaling not in _abi.ROTARY_SCALINGS:
            raise ValueError(f"scaling {scaling!r} is not one of {', '.join(_abi.ROTARY_SCALINGS)}")
        r = int(head_dim if rotary_dim is None else rotary_dim)
        if r > head_dim:
            raise ValueError(f"rotary_dim {r} is larger than head_dim {head_dim}")
        st, turns = _abi.dllm_rotary_frequencies(r, float(base), _abi.ROTARY_SCALINGS[scaling], float(factor),
                                                 int(original_len), float(fast), float(slow))
        if st != DLLM_OK:
            raise DllmError(st, "dllm_rotary_frequencies")
        if magnitude is None:
            magnitude = 0.1 * math.log(factor) + 1.0 if scaling == "ramp" else 1.0
        if not 0.0 < magnitude < 3e38:
            raise ValueError(f"magnitude {magnitude} is not a positive float32")
        self.head_dim, self.rotary_dim, self.magnitude = int(head_dim), r, float(magnitude)
        self.device = _device(device)
        self.stream = _stream(stream, self.device)
        self.turns = torch.tensor(turns, dtype=torch.float64, device=self.device)
        self.plan = _abi.dllm_rotary_plan(self.turns.data_ptr(), self.magnitude, r, _abi.ROTARY_LAYOUTS[layout])

    def __call__(self, x, positions, out=None, transpose: bool = False):
        """Queue out = x [T, H, head_dim] rotated to ``positions`` [T] (int32);
        returns out (new and contiguous unless given; may be x, but overlaps it
        in no other way).
        ``transpose`` turns the other way, which takes the gradient of the
        output to the gradient of x."""
        _heads(x, "x", None, self.head_dim, self.device)
        T, H, D = x.shape
        _need(positions, "positions", (torch.int32,), (T,), self.device)
        if out is not None:
            _heads(out, "out", H, D, self.device)
            if out.dtype != x.dtype or out.shape[0] != T:
                raise ValueError("out must have the type and shape of x")
        box = [out]

        def make(stream):
            y = box[0]
            if y is None:
                y = box[0] = x.new_empty((T, H, D))
            return _abi.load().dllm_rotary(C.byref(self.plan), x.data_ptr(), T, H, D, x.stride(0), x.stride(1),
                                           positions.data_ptr(), 1 if transpose else 0, y.data_ptr(), y.stride(0),
                                           y.stride(1), stream)

        self._call("dllm_rotary", (x, positions, out, self.turns), make)
        return box[0]


class CacheBatch:
    """The sequences of a call: ``cu`` [S + 1], ``lens`` [S] and ``table``
    [S, blocks] (int32, on the cache's device; include/dllm_cache.h).  The
    contents may change between calls, as a decoding loop's do; ``max_new``
    and ``max_len`` are host bounds on them (defaults: any number of new
    tokens, the table's whole capacity).  They choose kernels and size grids, so
    tight ones are faster: without ``max_new`` all new tokens of a call may be
    one sequence's."""

    def __init__(self, cu, lens, table, max_new: int | None, max_len: int | None, device):
        if table.dim() != 2 or table.shape[1] < 1:
            raise ValueError(f"table: shape {tuple(table.shape)}, expected [S, blocks]")
        S, blocks = table.shape
        if not 1 <= S <= 65535:
            raise ValueError(f"table: {S} sequences, 1 to 65535 are possible")
        i32 = (torch.int32,)
        _need(table, "table", i32, (S, blocks), device)
        _need(cu, "cu", i32, (S + 1,), device)
        _need(lens, "lens", i32, (S,), device)
        max_len = blocks * _BLOCK if max_len is None else int(max_len)
        if not 1 <= max_len <= blocks * _BLOCK:
            raise ValueError(f"max_len {max_len} is not in 1 .. {blocks * _BLOCK}, the table's capacity")
        if max_new is not None and int(max_new) < 1:
            raise ValueError(f"max_new {max_new} is not positive")
        self.S, self.blocks, self.max_len = int(S), int(blocks), max_len
        self.max_new = None if max_new is None else int(max_new)
        self.cu, self.lens, self.table, self.device = cu, lens, table, device
        self.struct = _abi.dllm_cache_batch(cu.data_ptr(), lens.data_ptr(), table.data_ptr(), self.S, self.blocks,
                                            self.max_new or (1 << 31) - 1, max_len)
        self._bytes = {}

    def _tensors(self):
        return self.cu, self.lens, self.table


class BlockCache(_Queued):
    """A pool of ``pages`` 32-token blocks of e4m3 keys and values for
    ``kv_heads`` heads of ``head_dim`` (64, 128 or 256), each block and head with
    power-of-two scales; include/dllm_cache.h gives the layout.  Which pages a
    sequence uses is the caller's: block tables name them."""

    def __init__(self, pages: int, kv_heads: int, head_dim: int, device="cuda", stream=None):
        dev = _device(device)
        u8 = dict(dtype=torch.uint8, device=dev)
        data = [torch.zeros((pages, kv_heads, _BLOCK * head_dim), **u8) for _ in range(2)]
        scale = [torch.full((pages, kv_heads), 127, **u8) for _ in range(2)]
        self._adopt(*data, *scale, stream)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream(dev))   # for these fills

    @classmethod
    def over(cls, k, v, k_scale, v_scale, stream=None) -> "BlockCache":
        """A cache over existing buffers: ``k``, ``v`` [pages, kv_heads,
        32 * head_dim] and ``k_scale``, ``v_scale`` [pages, kv_heads] (uint8)."""
        self = object.__new__(cls)
        self._adopt(k, v, k_scale, v_scale, stream)
        return self

    def _adopt(self, k, v, k_scale, v_scale, stream):
        if k.dim() != 3 or k.shape[2] % _BLOCK != 0 or k.shape[2] // _BLOCK not in (64, 128, 256):
            raise ValueError(f"k: shape {tuple(k.shape)}, expected [pages, kv_heads, 32 * head_dim] with a "
                             "head_dim of 64, 128 or 256")
        pages, heads, _ = k.shape
        if pages < 1 or heads < 1:
            raise ValueError("a cache has at least one page and one head")
        u8 = (torch.uint8,)
        _need(k, "k", u8, k.shape, k.device)
        _need(v, "v", u8, k.shape, k.device)
        _need(k_scale, "k_scale", u8, (pages, heads), k.device)
        _need(v_scale, "v_scale", u8, (pages, heads), k.device)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.pages, self.kv_heads, self.head_dim = int(pages), int(heads), int(k.shape[2]) // _BLOCK
        self.device, self.stream = k.device, _stream(stream, k.device)
        self.struct = _abi.dllm_cache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), self.pages,
                                      self.kv_heads, self.head_dim)

    def _buffers(self):
        return self.k, self.v, self.k_scale, self.v_scale

    def batch(self, cu, lens, table, max_new: int | None = None, max_len: int | None = None) -> CacheBatch:
        return CacheBatch(cu, lens, table, max_new, max_len, self.device)

    def _workspace(self, batch, name, *args):
        """Bytes of workspace: by sizes alone, so each is asked for once."""
        key = (name, self.kv_heads, self.head_dim, *args)
        nbytes = batch._bytes.get(key)
        if nbytes is None:
            nbytes = getattr(_abi, name)(self.struct, batch.struct, *args)
            if nbytes == 0:
                raise DllmError(DLLM_ERR_INVALID_ARG, name)
            batch._bytes[key] = nbytes
        return nbytes

    def _check_batch(self, batch):
        if not isinstance(batch, CacheBatch):
            raise TypeError("batch: a CacheBatch (BlockCache.batch) is expected")
        if batch.device != self.device:
            raise ValueError(f"batch: made for {batch.device}, expected {self.device}")

    def _queries(self, batch, q):
        self._check_batch(batch)
        _heads(q, "q", None, self.head_dim, self.device)
        if q.shape[1] < 1 or q.shape[1] % self.kv_heads != 0:
            raise ValueError(f"q: {q.shape[1]} heads, a multiple of {self.kv_heads} is expected")

    def write(self, batch: CacheBatch, k, v, start, positions=None, rotary: Rotary | None = None) -> None:
        """Queue the write of the new tokens' ``k`` and ``v`` [T, kv_heads,
        head_dim] (any strides) to slots ``start`` [S] onwards; ``rotary``
        rotates k to ``positions`` [T] first.  ``batch.lens`` counts the new
        tokens already."""
        self._check_batch(batch)
        _heads(k, "k", self.kv_heads, self.head_dim, self.device)
        _heads(v, "v", self.kv_heads, self.head_dim, self.device)
        T = k.shape[0]
        if v.shape[0] != T:
            raise ValueError(f"v: {v.shape[0]} tokens, k has {T}")
        _need(start, "start", (torch.int32,), (batch.S,), self.device)
        if (rotary is None) != (positions is None):
            raise ValueError("rotary and positions go together")
        plan = None
        if rotary is not None:
            _need(positions, "positions", (torch.int32,), (T,), self.device)
            if rotary.head_dim != self.head_dim or rotary.device != self.device:
                raise ValueError("rotary: made for another head_dim or device than the cache's")
            plan = C.byref(rotary.plan)

        def make(stream):
            return _abi.load().dllm_cache_write(
                C.byref(self.struct), C.byref(batch.struct), T, k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(),
                v.stride(0), v.stride(1), start.data_ptr(), positions.data_ptr() if positions is not None else None,
                plan, stream)

        self._call("dllm_cache_write", (k, v, start, positions, rotary.turns if rotary is not None else None,
                                        *self._buffers(), *batch._tensors()), make)

    def attend(self, batch: CacheBatch, q, scale: float | None = None, causal: bool = False, out=None, lse=False):
        """Queue attention of ``q`` [T, q_heads, head_dim] over the cache;
        returns out [T, q_heads, head_dim] (new unless given), or (out, lse)
        with ``lse`` True or a float32 [T, q_heads] tensor to fill.  ``scale``
        defaults to head_dim ** -0.5."""
        self._queries(batch, q)
        T, H, D = q.shape
        if scale is None:
            scale = D ** -0.5
        if out is not None:
            _need(out, "out", (q.dtype,), (T, H, D), self.device)
            if _overlap(q, out):
                raise ValueError("out: must not overlap q, which is read to the end")
        given = lse if isinstance(lse, torch.Tensor) else None
        if given is not None:
            _need(given, "lse", (torch.float32,), (T, H), self.device)
            if _overlap(q, given) or (out is not None and _overlap(out, given)):
                raise ValueError("lse: must not overlap q or out")
        want = given is not None or bool(lse)
        nbytes = self._workspace(batch, "dllm_cache_attention_workspace_bytes", H)
        box = [out, given]

        def make(stream):
            o, l = box
            if o is None:
                o = box[0] = q.new_empty((T, H, D))
            if l is None and want:
                l = box[1] = q.new_empty((T, H), dtype=torch.float32)
            ws = self.k.new_empty(nbytes)
            return _abi.load().dllm_cache_attention(
                C.byref(self.struct), C.byref(batch.struct), T, q.data_ptr(), q.stride(0), q.stride(1), H, scale,
                1 if causal else 0, o.data_ptr(), l.data_ptr() if l is not None else None, ws.data_ptr(), nbytes,
                stream)

        self._call("dllm_cache_attention", (q, out, given, *self._buffers(), *batch._tensors()), make)
        return (box[0], box[1]) if want else box[0]

    def weigh(self, batch: CacheBatch, q, lse, weights, scale: float | None = None, causal: bool = False,
              decay: float = 1.0) -> None:
        """Queue weights = decay * weights + the attention that each cached
        token received from ``q`` (``lse`` as attend returned it for the same
        arguments); ``weights`` [S, kv_heads, blocks * 32] float32."""
        self._queries(batch, q)
        T, H, D = q.shape
        if scale is None:
            scale = D ** -0.5
        _need(lse, "lse", (torch.float32,), (T, H), self.device)
        _need(weights, "weights", (torch.float32,), (batch.S, self.kv_heads, batch.blocks * _BLOCK), self.device)

        def make(stream):
            return _abi.load().dllm_cache_weigh(
                C.byref(self.struct), C.byref(batch.struct), T, q.data_ptr(), q.stride(0), q.stride(1), H, scale,
                1 if causal else 0, lse.data_ptr(), decay, weights.data_ptr(), stream)

        self._call("dllm_cache_weigh", (q, lse, weights, *self._buffers(), *batch._tensors()), make)

    def evict(self, batch: CacheBatch, weights, keep, table_out, sink: int = 0, recent: int = 0, pool: int = 1,
              lens_out=None, kept=None, weights_out=None):
        """Queue the eviction of all but ``keep`` [S] (int32) tokens of each
        sequence and head by their ``weights``, moving the kept ones to the
        pages of ``table_out`` [S, out_blocks].  ``kept`` [S, kv_heads,
        max_keep] receives their old places; its width bounds keep (default
        out_blocks * 32).  Returns (lens_out [S], kept, weights_out [S,
        kv_heads, out_blocks * 32]), new unless given; places behind a
        sequence's new length are not written."""
        self._check_batch(batch)
        S, H, dev = batch.S, self.kv_heads, self.device
        i32, f32 = (torch.int32,), (torch.float32,)
        _need(weights, "weights", f32, (S, H, batch.blocks * _BLOCK), dev)
        _need(keep, "keep", i32, (S,), dev)
        if table_out.dim() != 2 or table_out.shape[1] < 1:
            raise ValueError(f"table_out: shape {tuple(table_out.shape)}, expected [S, blocks]")
        blocks = int(table_out.shape[1])
        _need(table_out, "table_out", i32, (S, blocks), dev)
        if kept is not None and (kept.dim() != 3 or not 1 <= kept.shape[2] <= blocks * _BLOCK):
            raise ValueError(f"kept: shape {tuple(kept.shape)}, expected [S, kv_heads, 1 .. {blocks * _BLOCK}]")
        most = int(kept.shape[2]) if kept is not None else blocks * _BLOCK
        if kept is not None:
            _need(kept, "kept", i32, (S, H, most), dev)
        if lens_out is not None:
            _need(lens_out, "lens_out", i32, (S,), dev)
        if weights_out is not None:
            _need(weights_out, "weights_out", f32, (S, H, blocks * _BLOCK), dev)
        nbytes = self._workspace(batch, "dllm_cache_evict_workspace_bytes")
        box = [lens_out, kept, weights_out]

        def make(stream):
            if box[0] is None:
                box[0] = torch.empty(S, dtype=torch.int32, device=dev)
            if box[1] is None:
                box[1] = torch.empty((S, H, most), dtype=torch.int32, device=dev)
            if box[2] is None:
                box[2] = torch.empty((S, H, blocks * _BLOCK), dtype=torch.float32, device=dev)
            ws = self.k.new_empty(nbytes)
            return _abi.load().dllm_cache_evict(
                C.byref(self.struct), C.byref(batch.struct), weights.data_ptr(), keep.data_ptr(), most, sink, recent,
                pool, table_out.data_ptr(), blocks, box[0].data_ptr(), box[1].data_ptr(), box[2].data_ptr(),
                ws.data_ptr(), nbytes, stream)

        self._call("dllm_cache_evict", (weights, keep, table_out, lens_out, kept, weights_out, *self._buffers(),
                                        *batch._tensors()), make)
        return tuple(box)
