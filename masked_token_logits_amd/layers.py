"""The two ends of a masked diffusion model and what stands between its blocks,
with their gradients: the loss of the masked positions over the LM head, the
token embedding, and the residual update with its norms (include/dllm_loss.h,
dllm_embed.h, dllm_norm.h).

Streams as for the block cache: an object made with a stream queues on it,
without one each call queues on the stream that is current for its device;
what a call allocates belongs to the stream it runs on, and tensors passed to
a call on another stream than the current one are kept alive until that
stream is done with them.  Gradients are explicit calls; nothing is recorded.

Objects of another device than a GPU take their checks, but run nothing: a
valid call raises DLLM_ERR_UNSUPPORTED.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import _abi
from ._abi import DLLM_ERR_INVALID_ARG, DLLM_ERR_UNSUPPORTED, DllmError
from .cache import _BF16, _need, _Queued, _stream

_I32, _F32 = (torch.int32,), (torch.float32,)


def _at(t):
    return None if t is None else t.data_ptr()


def _rows(t, name: str, d: int, device) -> int:
    """[T, d] bf16; returns T."""
    if t.dim() != 2:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected [T, {d}]")
    _need(t, name, _BF16, (t.shape[0], d), device)
    return t.shape[0]


def _finite(x, name: str) -> float:
    x = float(x)
    if not abs(x) <= 3.4028234663852886e38:
        raise ValueError(f"{name} {x} is not a finite float32")
    return x


class _Workspace(_Queued):
    def _workspace(self, nbytes: int, where: str):
        if nbytes == 0:
            raise DllmError(DLLM_ERR_INVALID_ARG, where)
        return torch.empty(nbytes, dtype=torch.uint8, device=self.device)


class ResidualNorm(_Workspace):
    """The place between two blocks: x' = x + scale * gate * N(y, post) and
    n = N(x', pre), N(v, w) = w * v / sqrt(mean(v^2) + eps).

    ``pre``, ``post`` [d] bf16 weights of the norm before the next block and of
    the one behind the last; either may be None (no such norm).  Without both
    give ``d`` and ``device``."""

    def __init__(self, pre=None, post=None, eps: float = 1e-5, scale: float = 1.0, d: int | None = None, device=None,
                 stream=None):
        w = pre if pre is not None else post
        if w is not None:
            if w.dim() != 1:
                raise ValueError(f"weights: shape {tuple(w.shape)}, expected [d]")
            d = w.shape[0] if d is None else d
            device = w.device
        if d is None or device is None:
            raise ValueError("without pre and post, d and device are needed")
        self.d, self.device = int(d), torch.device(device)
        if self.device.type == "cuda" and self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        for t, name in ((pre, "pre"), (post, "post")):
            if t is not None:
                _need(t, name, _BF16, (self.d,), self.device)
        if self.d < 8 or self.d % 8 or self.d > _abi.DLLM_NORM_DIM_MAX:
            raise DllmError(DLLM_ERR_UNSUPPORTED, f"a norm of {self.d} dimensions")
        if not _finite(eps, "eps") >= 0:
            raise ValueError(f"eps {eps} is negative")
        self.pre, self.post, self.eps, self.scale = pre, post, float(eps), _finite(scale, "scale")
        self.stream = _stream(stream, self.device)
        self.struct = _abi.dllm_norm(_at(pre), _at(post), self.d, self.eps, self.scale)

    def _gate(self, gate, T: int) -> int:
        """The number of gate rows, 0 without a gate."""
        if gate is None:
            return 0
        if gate.dim() != 2 or gate.shape[0] < 1:
            raise ValueError(f"gate: shape {tuple(gate.shape)}, expected [groups, {self.d}]")
        G = gate.shape[0]
        _need(gate, "gate", _BF16, (G, self.d), self.device)
        if T % G or (G > 1 and T == 0):
            raise ValueError(f"gate: {T} tokens are not {G} equal runs")
        return G

    def __call__(self, x, y=None, gate=None, x_out=None, n_out=None):
        """Queue one update of x [T, d] by y [T, d]; returns (x', n), new unless
        given (``x_out`` may be x).  Without ``y`` x' is None and n = N(x, pre);
        without ``pre`` n is None.  ``gate`` [groups, d]: one row for each of
        ``groups`` equal runs of tokens."""
        T = _rows(x, "x", self.d, self.device)
        if y is None and (self.pre is None or self.post is not None or gate is not None or x_out is not None):
            raise ValueError("without y there is only the norm before a block")
        if self.pre is None and n_out is not None:
            raise ValueError("n_out: there is no norm before a block")
        for t, name in ((y, "y"), (x_out, "x_out"), (n_out, "n_out")):
            if t is not None:
                _need(t, name, _BF16, (T, self.d), self.device)
        groups, box = self._gate(gate, T), [x_out, n_out]

        def make(stream):
            if y is not None and box[0] is None:
                box[0] = torch.empty_like(x)
            if self.pre is not None and box[1] is None:
                box[1] = torch.empty_like(x)
            return _abi.load().dllm_residual_norm(C.byref(self.struct), x.data_ptr(), _at(y), T, _at(gate), groups,
                                                  _at(box[0]), _at(box[1]), stream)

        self._call("dllm_residual_norm", (x, y, gate, x_out, n_out, self.pre, self.post), make)
        return box[0], box[1]

    def backward(self, x, d_n=None, y=None, d_x=None, gate=None, d_x_out=None, d_y_out=None):
        """Queue the gradients of a call from those of its outputs: ``d_n`` of n
        and ``d_x`` of x' (either may be None: none), [T, d] bf16.  ``x`` is the
        stream behind the update, ``y`` and ``gate`` what the call had.

        Returns a dict: d_x and d_y [T, d] bf16 (``d_x_out``, ``d_y_out`` where
        given: they may be d_x or d_n, and y), d_pre and d_post [d] and
        d_gate [groups, d] float32; None for what the call did not have."""
        T = _rows(x, "x", self.d, self.device)
        if (d_n is None) != (self.pre is None):
            raise ValueError("d_n goes with the norm before a block")
        if d_n is None and d_x is None:
            raise ValueError("neither d_n nor d_x is given")
        if y is None and (self.post is not None or gate is not None or d_y_out is not None):
            raise ValueError("without y there is only the norm before a block")
        for t, name in ((y, "y"), (d_n, "d_n"), (d_x, "d_x"), (d_x_out, "d_x_out"), (d_y_out, "d_y_out")):
            if t is not None:
                _need(t, name, _BF16, (T, self.d), self.device)
        groups = self._gate(gate, T)
        got = dict(d_x=d_x_out, d_y=d_y_out, d_pre=None, d_post=None, d_gate=None)

        def make(stream):
            f32 = dict(dtype=torch.float32, device=self.device)
            new = torch.empty if T else torch.zeros     # no tokens, no launch: the sums are zero
            if got["d_x"] is None:
                got["d_x"] = torch.empty_like(x)
            if y is not None and got["d_y"] is None:
                got["d_y"] = torch.empty_like(y)
            if self.pre is not None:
                got["d_pre"] = new(self.d, **f32)
            if self.post is not None:
                got["d_post"] = new(self.d, **f32)
            if groups:
                got["d_gate"] = new((groups, self.d), **f32)
            lib = _abi.load()
            nbytes = lib.dllm_residual_norm_backward_workspace_bytes(C.byref(self.struct), T, groups)
            ws = self._workspace(nbytes, "dllm_residual_norm_backward_workspace_bytes")
            return lib.dllm_residual_norm_backward(
                C.byref(self.struct), x.data_ptr(), _at(y), T, _at(gate), groups, _at(d_n), _at(d_x), _at(got["d_x"]),
                _at(got["d_y"]), _at(got["d_pre"]), _at(got["d_post"]), _at(got["d_gate"]), ws.data_ptr(), nbytes, stream)

        self._call("dllm_residual_norm_backward", (x, y, gate, d_n, d_x, d_x_out, d_y_out, self.pre, self.post), make)
        return got


class Embedding(_Workspace):
    """Rows of ``table`` [V, d] (bf16) by token, times ``scale``.  A token
    outside 0 .. V - 1 has no row: its output is zero, and it adds to no
    gradient."""

    def __init__(self, table, scale: float = 1.0, stream=None):
        if table.dim() != 2 or table.shape[0] < 1:
            raise ValueError(f"table: shape {tuple(table.shape)}, expected [V, d]")
        self.V, self.d = map(int, table.shape)
        self.device = table.device
        _need(table, "table", _BF16, (self.V, self.d), self.device)
        if self.d < 8 or self.d % 8:
            raise DllmError(DLLM_ERR_UNSUPPORTED, f"an embedding of {self.d} dimensions")
        self.table, self.scale, self.stream = table, _finite(scale, "scale"), _stream(stream, self.device)

    def _tokens(self, tokens) -> int:
        if tokens.dim() != 1:
            raise ValueError(f"tokens: shape {tuple(tokens.shape)}, expected [T]")
        _need(tokens, "tokens", _I32, tokens.shape, self.device)
        return tokens.shape[0]

    def __call__(self, tokens, out=None):
        """Queue out [T, d] = scale * table[tokens [T] int32]; returns out (new unless given)."""
        T, box = self._tokens(tokens), [out]
        if out is not None:
            _need(out, "out", _BF16, (T, self.d), self.device)

        def make(stream):
            if box[0] is None:
                box[0] = self.table.new_empty((T, self.d))
            return _abi.load().dllm_embed(self.table.data_ptr(), self.V, self.d, tokens.data_ptr(), T, self.scale,
                                          box[0].data_ptr(), stream)

        self._call("dllm_embed", (tokens, out, self.table), make)
        return box[0]

    def backward(self, tokens, d_out, d_table=None, accumulate: bool = False):
        """Queue the table's gradient [V, d] (bf16) from that of the output,
        ``d_out`` [T, d]; returns it.  ``accumulate`` adds it to what the given
        ``d_table`` holds and touches only rows of tokens that occur."""
        T, box = self._tokens(tokens), [d_table]
        _need(d_out, "d_out", _BF16, (T, self.d), self.device)
        if d_table is not None:
            _need(d_table, "d_table", _BF16, (self.V, self.d), self.device)
        elif accumulate:
            raise ValueError("accumulate needs the d_table to add to")

        def make(stream):
            if box[0] is None:
                box[0] = torch.empty_like(self.table)
            lib = _abi.load()
            nbytes = lib.dllm_embed_backward_workspace_bytes(self.V, self.d, T)
            ws = self._workspace(nbytes, "dllm_embed_backward_workspace_bytes")
            return lib.dllm_embed_backward(tokens.data_ptr(), T, d_out.data_ptr(), self.V, self.d, self.scale,
                                           1 if accumulate else 0, box[0].data_ptr(), ws.data_ptr(), nbytes, stream)

        self._call("dllm_embed_backward", (tokens, d_out, d_table), make)
        return box[0]


class MaskedLoss(_Workspace):
    """Cross entropy of the masked positions over the LM head ``W_lm`` [V, d]
    (bf16), without the logits.  A position counts where ``mask`` is not zero
    and its target is a token (0 .. V - 1).

    ``piece``: vocabulary entries whose gradient of the logits the backward
    pass holds at a time (a multiple of 256; None: about 1 GiB's worth)."""

    def __init__(self, W_lm, piece: int | None = None, stream=None):
        if W_lm.dim() != 2 or W_lm.shape[0] < 1:
            raise ValueError(f"W_lm: shape {tuple(W_lm.shape)}, expected [V, d]")
        self.V, self.d = map(int, W_lm.shape)
        self.device = W_lm.device
        _need(W_lm, "W_lm", _BF16, (self.V, self.d), self.device)
        if self.d < 8 or self.d % 8:
            raise DllmError(DLLM_ERR_UNSUPPORTED, f"a head of {self.d} dimensions")
        if piece is not None and (int(piece) < 256 or int(piece) % 256):
            raise ValueError(f"piece {piece} is not a positive multiple of 256")
        self.W_lm, self.piece, self.stream = W_lm, int(piece or 0), _stream(stream, self.device)
        self._bytes = {}     # workspace sizes of the lengths seen: (forward, backward)

    def _struct(self, hidden, mask, targets, weights):
        L = _rows(hidden, "hidden", self.d, self.device)
        if L < 1:
            raise ValueError("hidden: no positions")
        _need(mask, "mask", (torch.uint8, torch.bool), (L,), self.device)
        _need(targets, "targets", _I32, (L,), self.device)
        if weights is not None:
            _need(weights, "weights", _F32, (L,), self.device)
        return _abi.dllm_loss(self.W_lm.data_ptr(), hidden.data_ptr(), mask.data_ptr(), targets.data_ptr(),
                              _at(weights), self.V, self.d, L)

    def _workspaces(self, L: int):
        got = self._bytes.get(L)
        if got is None:
            got = self._bytes[L] = (_abi.dllm_loss_forward_workspace_bytes(self.V, self.d, L),
                                    _abi.dllm_loss_backward_workspace_bytes(self.V, self.d, L, self.piece))
        return got

    def __call__(self, hidden, mask, targets, weights=None, out=None):
        """Queue the loss of hidden [L, d] at the masked positions (mask [L] u8
        or bool, targets [L] int32, weights [L] float32 or None = 1).

        Returns (loss [1], losses [L], lse [L]) float32: the weighted sum, each
        position's cross entropy and log-sum-exp (0 where it does not count);
        ``out`` gives the three buffers."""
        p = self._struct(hidden, mask, targets, weights)
        L = p.L
        box = list(out) if out is not None else None
        if box is not None:
            if len(box) != 3:
                raise ValueError("out is (loss, losses, lse)")
            for t, name, n in zip(box, ("loss", "losses", "lse"), (1, L, L)):
                _need(t, name, _F32, (n,), self.device)

        def make(stream):
            nonlocal box
            if box is None:
                new = self.W_lm.new_empty
                box = [new((n,), dtype=torch.float32) for n in (1, L, L)]
            nbytes = self._workspaces(L)[0]
            ws = self._workspace(nbytes, "dllm_loss_forward_workspace_bytes")
            return _abi.load().dllm_loss_forward(C.byref(p), box[0].data_ptr(), box[1].data_ptr(), box[2].data_ptr(),
                                                 ws.data_ptr(), nbytes, stream)

        self._call("dllm_loss_forward", (hidden, mask, targets, weights, self.W_lm, *(box or ())), make)
        return tuple(box)

    def backward(self, hidden, mask, targets, lse, weights=None, grad=None, d_hidden=None, d_W=None,
                 accumulate: bool = False, need=("hidden", "W")):
        """Queue the gradients of a loss call with the same inputs; ``lse`` is
        what it returned and ``grad`` [1] float32 the gradient of the loss
        (None: 1).

        Returns (d_hidden [L, d], d_W [V, d]) bf16, new unless given; ``need``
        names those that are wanted, the other is None.  ``accumulate`` adds to
        what the given ``d_W`` holds."""
        p = self._struct(hidden, mask, targets, weights)
        L = p.L
        need = set(need) | ({"hidden"} if d_hidden is not None else set()) | ({"W"} if d_W is not None else set())
        if not need or need - {"hidden", "W"}:
            raise ValueError("need names hidden, W or both")
        _need(lse, "lse", _F32, (L,), self.device)
        if grad is not None:
            _need(grad, "grad", _F32, (1,), self.device)
        if d_hidden is not None:
            _need(d_hidden, "d_hidden", _BF16, (L, self.d), self.device)
        if d_W is not None:
            _need(d_W, "d_W", _BF16, (self.V, self.d), self.device)
        elif accumulate:
            raise ValueError("accumulate needs the d_W to add to")
        box = [d_hidden, d_W]

        def make(stream):
            if box[0] is None and "hidden" in need:
                box[0] = torch.empty_like(hidden)
            if box[1] is None and "W" in need:
                box[1] = torch.empty_like(self.W_lm)
            nbytes = self._workspaces(L)[1]
            ws = self._workspace(nbytes, "dllm_loss_backward_workspace_bytes")
            return _abi.load().dllm_loss_backward(C.byref(p), lse.data_ptr(), _at(grad), _at(box[0]), _at(box[1]),
                                                  1 if accumulate else 0, self.piece, ws.data_ptr(), nbytes, stream)

        self._call("dllm_loss_backward", (hidden, mask, targets, lse, weights, grad, d_hidden, d_W, self.W_lm), make)
        return box[0], box[1]
